"""8-bit-float layers on the GPU against plain float64 forms.

Bytes and scales of the quantisers are exact: a scale is a power of two and
the only rounding is the one to e4m3. Where the rounded value itself is formed
in fp32 (swiglu, rmsnorm) its relative error is at most DELTA, so a byte may be
that of any value within DELTA of the exact one, and nothing else; the scales
still have to be equal.

The products are held to (64 + KB) 2^-24 sum |x||w| (KB blocks of K): every
block's partial sum is added with one fp32 rounding of a running sum that is
at most sum |x||w| (KB roundings, and two for the scales), and inside a block
each of the four 32-deep steps of the tensor cores may lose a few units in the
last place of fp32, for which 64 units are ample. bf16 outputs add half a bf16
step, 2^-8 |y|.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

# h = t * rstd * g: the root (2 ulp), the cast of the mean and two products;
# silu(g) * u: the exponential (2 ulp), sum, quotient and product. 16 half-steps cover both.
DELTA = 16 * 2.0 ** -24
E4M3 = np.array([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)][:127])


def to_e4m3(v):
    """Nearest entry of the table of the 127 magnitudes; ties to the even code."""
    mag = np.abs(v)
    i = np.clip(np.searchsorted(E4M3, mag), 1, 126)
    lo, hi = E4M3[i - 1], E4M3[i]
    up = (mag - lo > hi - mag) | ((mag - lo == hi - mag) & (i % 2 == 0))
    code = np.where(up, i, i - 1).astype(np.int64)
    code = np.where(np.signbit(v), code + 128, code)
    return np.where(np.isnan(v), 127, code).astype(np.uint8)


def scale_of(amax):
    out = np.ones_like(amax)
    for idx in np.ndindex(amax.shape):
        a = float(amax[idx])
        if a > 0:
            e = -126
            while a > 448.0 * 2.0 ** e and e < 120:
                e += 1
            out[idx] = 2.0 ** e
    return out


def ref_scales(h, rows=1):
    """Scales of blocks of rows x 128 of a float64 matrix, NaN left out, infinities as the largest float."""
    M, K = h.shape
    a = np.nan_to_num(np.abs(h), nan=0.0, posinf=3.402823466e38)
    nb, kb = -(-M // rows), -(-K // 128)
    p = np.zeros((nb * rows, kb * 128))
    p[:M, :K] = a
    return scale_of(p.reshape(nb, rows, kb, 128).max(axis=(1, 3)))


def spread_scales(s, M, K, rows=1):
    return np.repeat(np.repeat(s, rows, 0)[:M], 128, 1)[:, :K]


def f64(t):
    return t.detach().double().cpu().numpy()


def codes(q):
    import torch
    return q.view(torch.uint8).cpu().numpy()


def check_bytes(q, scales, h, K, delta=0.0, rows=1, exact_scales=True):
    """q and scales against the float64 matrix h."""
    M = h.shape[0]
    s = ref_scales(h, rows)
    got_s = f64(scales)
    if exact_scales:
        assert np.array_equal(got_s, s), np.argwhere(got_s != s)[:5]
    full = spread_scales(s, M, K, rows)
    got = codes(q)
    if rows == 1:
        assert got.shape == (M, -(-K // 16) * 16)
        assert not got[:, K:].any(), "padding is not zero"
    got = got[:, :K]
    with np.errstate(invalid="ignore"):
        v = np.where(np.isinf(h), np.nan, h) / full
    lo, hi = to_e4m3(v * (1 - delta)), to_e4m3(v * (1 + delta))
    nan = np.isnan(v)
    assert np.array_equal((got & 0x7F) == 0x7F, nan)
    zero = ((got & 0x7F) == 0) & ((lo & 0x7F) == 0)  # either zero
    ok = (got == lo) | (got == hi) | nan | zero
    assert ok.all(), (np.argwhere(~ok)[:3], h[~ok][:3], got[~ok][:3], lo[~ok][:3])


def randn(seed, *shape, scale=1.0):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, device="cuda", generator=g) * scale


def dtype(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def unaligned(t):
    """The same values at an address one element past a 16-byte boundary."""
    import torch
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    flat[1:] = t.reshape(-1)
    return flat[1:].view(t.shape)


# ---- quantisers -------------------------------------------------------------------

SHAPES = [(1, 1), (1, 16), (1, 127), (1, 128), (2, 129), (3, 200), (5, 2048), (37, 1000), (2, 16401), (300, 384)]


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_quantize(hxq, M, K, dt):
    x = randn(M * 7919 + K, M, K, scale=3.0).to(dtype(dt))
    for t in (x, unaligned(x)):
        q, s = hxq.fp8_quantize(t)
        check_bytes(q, s, f64(x), K)


def test_quantize_special_values(hxq):
    import torch
    x = randn(5, 16, 256)
    x[0] = 0
    x[1, :128] = 0
    x[2, 5] = float("nan")
    x[3, 200] = float("inf")
    x[3, 201] = -float("inf")
    x[4] = x[4] * 1e-42          # subnormal floats
    x[5] = x[5] * 1e38
    x[6, :128] = torch.linspace(-448, 448, 128)
    x[7, :128] = torch.nextafter(torch.tensor(448.0), torch.tensor(1e9)).item()
    x[8, 0], x[8, 1:128] = 448.0, torch.tensor([17.0, 19.0, -21.0, 0.0009765625, 0.0029296875, -0.0] * 22)[:127].cuda()
    x[9] = float("nan")
    x[10, 0] = 3.4e38
    for t in (x, x.to(torch.bfloat16)):
        q, s = hxq.fp8_quantize(t)
        check_bytes(q, s, f64(t), 256)


def test_quantize_ties_to_even(hxq):
    """Every midpoint of two neighbouring e4m3 values, in a block whose scale is 1."""
    import torch
    mids = (E4M3[:-1] + E4M3[1:]) / 2
    x = torch.zeros(2, 128)
    x[0, 0], x[0, 1:127] = 448.0, torch.tensor(mids, dtype=torch.float32)
    x[1] = -x[0]
    q, s = hxq.fp8_quantize(x.cuda())
    check_bytes(q, s, f64(x), 128)
    assert (codes(q)[0, 1:127] % 2 == 0).all()


@pytest.mark.parametrize("N,K,E", [(1, 1, 1), (128, 128, 1), (129, 130, 1), (300, 200, 3), (64, 1001, 2), (512, 640, 1)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_encode(hxq, N, K, E, dt):
    W = randn(N + K, E, N, K, scale=0.02).to(dtype(dt))
    W[0, 0, 0] = 1.0
    for t in (W, unaligned(W)):
        q, s = hxq.fp8_encode(t)
        assert q.shape == W.shape
        for e in range(E):
            check_bytes(q[e], s[e], f64(W[e]), K, rows=128)


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_swiglu(hxq, M, K, dt):
    gu = randn(M + 31 * K, M, 2 * K, scale=4.0).to(dtype(dt))
    g, u = f64(gu[:, :K]), f64(gu[:, K:])
    h = g / (1 + np.exp(-g)) * u
    for t in (gu, unaligned(gu)):
        q, s = hxq.fp8_swiglu(t)
        check_bytes(q, s, h, K, DELTA)


def test_swiglu_extremes(hxq):
    """Gates whose exponential over- or underflows, and blocks of tiny values only."""
    import torch
    gu = randn(3, 6, 512)
    gu[0, :256] = -80.0
    gu[1, :256] = 120.0
    gu[2, :256] = -torch.linspace(60, 100, 256).cuda()
    gu[3, :256] = 0.0
    gu[4, 7] = float("nan")
    gu[5, :256] = -200.0
    g, u = f64(gu[:, :256]), f64(gu[:, 256:])
    with np.errstate(over="ignore"):
        h = g / (1 + np.exp(-g)) * u
    q, s = hxq.fp8_swiglu(gu)
    check_bytes(q, s, h, 256, DELTA)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("K", [256, 250])
def test_swiglu_low_gates_large_ups(hxq, dt, K):
    """Gates at and below -87, where e^-g nears the end of fp32, beside ups that keep the value large."""
    import torch
    gu = randn(3, 6, 2 * K)
    gu[0, :K] = -torch.linspace(80, 95, K).cuda()
    gu[0, K:] = 3e38
    gu[1, 5], gu[1, K + 5] = -88.0, 3e38
    gu[2, 6], gu[2, K + 6] = -300.0, -3e38
    gu[3, :K] = -88.5
    gu[4, 9], gu[4, K + 9] = -87.0, 3e38
    gu[5, 9], gu[5, K + 9] = -104.0, -3e38
    gu = gu.to(dtype(dt))
    g, u = f64(gu[:, :K]), f64(gu[:, K:])
    h = g / (1 + np.exp(-g)) * u
    q, s = hxq.fp8_swiglu(gu)
    check_bytes(q, s, h, K, DELTA)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("K", [256, 250])
def test_swiglu_ends_of_range(hxq, dt, K):
    """Gates near fp32's largest, infinite and below its normal numbers, beside small and large ups."""
    import torch
    inf = float("inf")
    gu = randn(4, 8, 2 * K)
    gu[0, 5], gu[0, K + 5] = 3e38, 1e-38
    gu[1, 5], gu[1, K + 5] = 3e38, 1.0
    gu[2, 5], gu[2, K + 5] = 3e38, 3e38
    gu[3, 5], gu[3, K + 5] = inf, -1.0
    gu[4, 5], gu[4, K + 5] = -inf, 1.0
    gu[5, :K], gu[5, K:] = 3 * 2.0 ** -133, 2.0 ** 127
    gu[5, 5], gu[5, K + 5] = 1.0, 2.0 ** -6
    gu[6, 5], gu[6, K + 5] = 1.0, inf
    gu[7, 5], gu[7, K + 5] = -60.0, 3e38
    gu = gu.to(dtype(dt))
    g, u = f64(gu[:, :K]), f64(gu[:, K:])
    with np.errstate(over="ignore", invalid="ignore"):
        h = g / (1 + np.exp(-g)) * u
    h[np.abs(h) > np.finfo(np.float32).max] = inf  # beyond fp32 it counts as infinite
    q, s = hxq.fp8_swiglu(gu)
    check_bytes(q, s, h, K, DELTA)


# ---- norm -------------------------------------------------------------------------

def ref_norm(x, res, w, eps):
    """(t as a tensor, h in float64)."""
    t = x if res is None else (x.float() + res.float()).to(res.dtype)
    d = f64(t)
    with np.errstate(invalid="ignore", divide="ignore"):
        h = d / np.sqrt((d * d).mean(1, keepdims=True) + eps)
    return t, h * f64(w) if w is not None else h


def check_y(y, h):
    y = f64(y)
    assert np.array_equal(np.isnan(y), np.isnan(h))
    ok = np.isnan(h) | (np.abs(y - h) <= (2.0 ** -8 + DELTA) * np.abs(h) + 2.0 ** -133)  # (2^-133: a bf16 subnormal step)
    assert ok.all(), (np.argwhere(~ok)[:3], y[~ok][:3], h[~ok][:3])


NORM_SHAPES = [(1, 1), (1, 130), (3, 8), (7, 200), (2, 2048), (5, 3584), (2, 4104), (3, 8200), (2, 14336), (1, 16384),
               (2, 32768), (1, 33000), (2, 40001), (1, 100000)]


@pytest.mark.parametrize("M,K", NORM_SHAPES)
@pytest.mark.parametrize("xt,rt", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_rmsnorm(hxq, M, K, xt, rt):
    import torch
    x = randn(M + K, M, K).to(dtype(xt))
    res = randn(M + K + 1, M, K, scale=5.0).to(dtype(rt))
    w = 1 + randn(M + K + 2, K, scale=0.2)
    t, h = ref_norm(x, res, w, 1e-5)
    for xx, rr, ww in ((unaligned(x), unaligned(res), unaligned(w)), (x, res, w)):
        q, s, y, total = hxq.rmsnorm(xx, ww, 1e-5, residual=rr, want="qy")
        assert torch.equal(total, t)
        check_bytes(q, s, h, K, DELTA)
        check_y(y, h)
    # one output alone gives the same, and the sum may replace the residual
    q1, s1, y1, _ = hxq.rmsnorm(x, w, 1e-5, residual=res)
    assert y1 is None and torch.equal(codes_t(q1), codes_t(q)) and torch.equal(s1, s)
    own = res.clone()
    _, _, y2, total2 = hxq.rmsnorm(x, w, 1e-5, residual=own, sum_out=own, want="y")
    assert total2.data_ptr() == own.data_ptr() and torch.equal(own, t) and torch.equal(y2, y)


def codes_t(q):
    import torch
    return q.view(torch.uint8)


@pytest.mark.parametrize("xt", ["f32", "bf16"])
def test_rmsnorm_without_residual_or_weight(hxq, xt):
    x = randn(9, 4, 1000).to(dtype(xt))
    _, h = ref_norm(x, None, None, 1e-6)
    q, s, y, total = hxq.rmsnorm(x, want="qy")
    assert total is None
    check_bytes(q, s, h, 1000, DELTA)
    check_y(y, h)


@pytest.mark.parametrize("xt", ["f32", "bf16"])
def test_rmsnorm_extremes(hxq, xt):
    """Rows of zeros, of values whose squares leave fp32's range, and with NaN or infinity; neighbours keep theirs."""
    x = randn(10, 8, 384)
    x[0] = 0
    x[1] *= 1e25
    x[2] *= 1e-30
    x[3, 5] = float("nan")
    x[4, 6] = float("inf")
    x[6] *= 3e37
    x = x.to(dtype(xt))
    w = 1 + randn(11, 384, scale=0.1)
    w[128:256] = 0
    _, h = ref_norm(x, None, w, 0.0)
    _, h1 = ref_norm(x, None, w, 1e-6)
    q, s, y, _ = hxq.rmsnorm(x, w, 1e-6, want="qy")
    keep = [0, 1, 2, 5, 6, 7]
    check_bytes(q[keep], s[keep], h1[keep], 384, DELTA)
    check_y(y[keep], h1[keep])
    assert np.isnan(f64(y)[3]).all() and ((codes(q)[3] & 0x7F) == 0x7F).all()
    assert (f64(s)[3] == 1).all()  # nothing but NaN: no maximum
    yi = f64(y)[4]  # the root is infinite: inf / inf is NaN and the others are 0
    assert np.isnan(yi[6]) and (np.delete(yi, 6) == 0).all()
    assert (codes(q)[4, 6] & 0x7F) == 0x7F and not (np.delete(codes(q)[4], 6) & 0x7F).any()
    q0, s0, y0, _ = hxq.rmsnorm(x, w, 0.0, want="qy")
    assert np.isnan(f64(y0)[0]).all() and (f64(s0)[0] == 1).all()  # 0 / 0, as the formula says
    check_y(y0[keep[1:]], h[keep[1:]])
    check_bytes(q0[keep[1:]], s0[keep[1:]], h[keep[1:]], 384, DELTA)


@pytest.mark.parametrize("xt,K", [("f32", 256), ("bf16", 256), ("f32", 20000), ("bf16", 20000), ("bf16", 3592)])
def test_rmsnorm_scales_at_their_borders(hxq, xt, K):
    """Rows whose largest |h| is 448 s, or a few roundings of fp32 away from it: the scale is the one of the exact h.
    Row r's largest value is in column r, whose weight is aimed at the border and nudged."""
    import torch
    rows = 64
    x = randn(12, rows, K)
    x[torch.arange(rows), torch.arange(rows)] = 60.0 + torch.rand(rows, device="cuda")
    x = x.to(dtype(xt))
    w = 1 + randn(13, K, scale=0.1)
    # the other rows' aimed columns are 0
    col, row = torch.arange(K, device="cuda")[None], torch.arange(rows, device="cuda")[:, None]
    x = torch.where((col < rows) & (col != row), torch.zeros_like(x), x)
    d = f64(x)
    root = np.sqrt((d * d).mean(1))
    for r in range(rows):
        g = np.float32(14.0 * root[r] / d[r, r])  # 14 = 448 / 32
        for _ in range(abs(r % 9 - 4)):
            g = np.nextafter(g, np.float32(np.inf if r % 9 > 4 else -np.inf))
        w[r] = float(g)
    _, h = ref_norm(x, None, w, 0.0)
    assert (np.abs(h[np.arange(rows), np.arange(rows)] / 14.0 - 1) < 1e-6).all()
    assert len(set(ref_scales(h)[:, 0])) == 2
    q, s, _, _ = hxq.rmsnorm(x, w, 0.0)
    check_bytes(q, s, h, K, DELTA)


def test_other_layouts_are_copied(hxq):
    """A transposed and a sliced input give what their contiguous copies give, on the current stream and on another,
    by object and by handle, whose work before the call the copy waits for."""
    import torch
    base = randn(3, 200, 300)
    st = torch.cuda.Stream()
    for x in (base.t(), base[:, 7:263], base[::2]):
        for f in (hxq.fp8_quantize, hxq.fp8_encode, lambda v, **k: hxq.rmsnorm(v, **k)[:2]):
            a, b = f(x), f(x.contiguous())
            assert torch.equal(codes_t(a[0]), codes_t(b[0])) and torch.equal(a[1], b[1])
            keep = base.clone()
            for handle in (st, st.cuda_stream):
                base.zero_()
                st.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(st):
                    base.copy_(keep)
                c = f(x, stream=handle)
                st.synchronize()
                assert torch.equal(codes_t(a[0]), codes_t(c[0])) and torch.equal(a[1], c[1])


def test_row_operators_on_another_stream_and_captured(hxq):
    """Each of them on a stream of its own behind the work that fills its input there, eager and as a graph."""
    import torch
    src = randn(4, 300, 1024)
    x = torch.empty_like(src)
    res = randn(5, 300, 1024)
    calls = [lambda s: hxq.fp8_quantize(x, stream=s), lambda s: hxq.fp8_swiglu(x, stream=s),
             lambda s: hxq.fp8_encode(x, stream=s), lambda s: hxq.rmsnorm(x, residual=res, want="qy", stream=s)]
    x.copy_(src)
    want = [[t.clone() for t in c(None) if t is not None] for c in calls]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    same = lambda a, b: torch.equal(a.view(torch.uint8), b.view(torch.uint8))  # noqa: E731
    for c, w in zip(calls, want):
        x.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            x.copy_(src)
            got = [t for t in c(st) if t is not None]
        st.synchronize()
        assert all(same(a, b) for a, b in zip(got, w))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            x.copy_(src)
            got = [t for t in c(None) if t is not None]
        x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, w))


# ---- products -----------------------------------------------------------------------

def make_activation(seed, M, K):
    """8-bit values and scales that no quantiser made: any fp32 scale."""
    import torch
    ld = -(-K // 16) * 16
    q = randn(seed, M, ld, scale=100.0).clamp_(-448, 448).to(torch.float8_e4m3fn)
    s = 0.01 * torch.exp(randn(seed + 1, M, -(-K // 128)))
    return q, s


def make_weights(seed, E, N, K):
    import torch
    q = randn(seed, E, N, K, scale=100.0).clamp_(-448, 448).to(torch.float8_e4m3fn)
    s = 3e-4 * torch.exp(randn(seed + 1, E, -(-N // 128), -(-K // 128)))
    return q, s


def dense_x(q, s, K):
    return q[:, :K].double() * s.double().repeat_interleave(128, 1)[:, :K]


def dense_w(q, s):
    N, K = q.shape
    return q.double() * s.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]


def check_product(y, x, w, bias, what=""):
    """y against float64 x . w^T + bias."""
    import torch
    ref = x @ w.t()
    scale = x.abs() @ w.abs().t()
    kb = -(-x.shape[1] // 128)
    if bias is not None:
        ref = ref + bias.double()
        scale = scale + bias.double().abs()
    tol = (64 + kb) * 2.0 ** -24 * scale
    if y.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * ref.abs()
    err = (y.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}; first {bad.nonzero()[:3].tolist()} " \
                          f"y {y[bad][:3].tolist()} ref {ref[bad][:3].tolist()}"


LINEAR = [
    # (M, N, K)
    (1, 1, 1), (1, 128, 128), (1, 2048, 2048), (1, 130, 1000), (2, 256, 131), (3, 8512, 2048), (7, 300, 40),
    (16, 2048, 4096), (17, 640, 1152), (29, 2048, 11008), (32, 500, 2048), (33, 257, 129), (48, 1024, 3584),
    (64, 11008, 512), (65, 384, 640), (100, 1000, 1000), (128, 2048, 2048), (129, 130, 270), (200, 896, 3584),
    (255, 512, 256), (256, 2048, 512), (257, 3584, 384), (512, 1920, 1024), (513, 1000, 2000), (1000, 2816, 1408),
    (2048, 3584, 512), (1, 300, 20000), (130, 300, 20000), (4097, 300, 264),
]


@pytest.mark.parametrize("M,N,K", LINEAR)
def test_linear(hxq, M, N, K):
    import torch
    xq, xs = make_activation(M + N, M, K)
    wq, ws = make_weights(N + K, 1, N, K)
    bias = randn(77, N)
    x, w = dense_x(xq, xs, K), dense_w(wq[0], ws[0])
    lin = hxq.Fp8Linear(wq[0], ws[0])
    for out, b in ((hxq.HXQ_OUT_F32, None), (hxq.HXQ_OUT_BF16, bias), (hxq.HXQ_OUT_F32, bias), (hxq.HXQ_OUT_BF16, None)):
        # the buffers end with guard rows, which no call may touch
        dt = torch.bfloat16 if out == hxq.HXQ_OUT_BF16 else torch.float32
        buf = torch.full((M + 2, N), 7.0, dtype=dt, device="cuda")
        y = lin.forward(xq, xs, bias=b, out_dtype=out, y=buf[1:M + 1])
        check_product(y, x, w, b, f"M={M} N={N} K={K} out={out}")
        assert (buf[0] == 7).all() and (buf[-1] == 7).all()
        assert torch.equal(lin.forward(xq, xs, bias=b, out_dtype=out), y)  # bitwise repeatable
    lin.check()


@pytest.mark.parametrize("M", [1, 20, 128, 300])
def test_a_row_does_not_depend_on_the_others(hxq, M):
    """NaN in one token's bytes or scales, and whatever lies behind the last row, reach no other row."""
    import torch
    N, K = 260, 700
    q, s = make_activation(5, M + 40, K)
    wq, ws = make_weights(6, 1, N, K)
    lin = hxq.Fp8Linear(wq[0], ws[0])
    y0 = lin.forward(q[:M], s[:M])
    q2, s2 = q.clone(), s.clone()
    codes_t(q2)[M:] = 0x7F
    s2[M:] = float("nan")
    assert torch.equal(lin.forward(q2[:M], s2[:M]), y0)
    if M > 1:
        codes_t(q2)[M // 2] = 0x7F
        s2[0] = float("nan")
        y1 = lin.forward(q2[:M], s2[:M])
        keep = [i for i in range(M) if i not in (0, M // 2)]
        assert torch.equal(y1[keep], y0[keep])
        assert y1[0].isnan().all() and y1[M // 2].isnan().all()
    # bytes between K and the row's end are not read
    codes_t(q2)[:] = codes_t(q)
    codes_t(q2)[:, K:] = 0x7F
    assert torch.equal(lin.forward(q2[:M], s[:M]), y0)


def test_extreme_scales(hxq):
    """Scales near both ends of fp32 whose product is ordinary."""
    import torch
    xq, xs = make_activation(1, 40, 384)
    wq, ws = make_weights(2, 1, 200, 384)
    y = hxq.Fp8Linear(wq[0], ws[0] * 2.0 ** 100).forward(xq, xs * 2.0 ** -100)
    assert torch.equal(y, hxq.Fp8Linear(wq[0], ws[0]).forward(xq, xs))


@pytest.mark.parametrize("M", [1, 24, 60, 500])
@pytest.mark.parametrize("e", [-112, 112])
def test_scales_at_the_ends_of_fp32(hxq, M, e):
    """Products times one scale alone would over- or underflow; times both they are ordinary."""
    import torch
    xq, xs = make_activation(1, M, 640)
    wq, ws = make_weights(2, 1, 200, 640)
    # (powers of two near 1, so that none of the scales itself leaves fp32)
    xs = 2.0 ** torch.randint(-2, 3, xs.shape, device="cuda").float()
    ws = 2.0 ** torch.randint(-2, 3, ws.shape, device="cuda").float()
    want = hxq.Fp8Linear(wq[0], ws[0]).forward(xq, xs)
    assert torch.isfinite(want).all() and want.abs().max() > 2.0 ** 16
    y = hxq.Fp8Linear(wq[0], ws[0] * 2.0 ** -e).forward(xq, xs * 2.0 ** e)
    assert torch.equal(y, want)


def offsets_of(counts, first=0):
    import torch
    return torch.tensor(np.concatenate([[first], first + np.cumsum(counts)]), dtype=torch.int32, device="cuda")


GROUPED = [
    # (rows per expert, rows in front, rows behind, N, K)
    ([1], 0, 0, 128, 128),
    ([0, 1, 0], 0, 0, 130, 200),
    ([3, 0, 5, 16, 1, 0, 7], 0, 0, 300, 1000),
    ([2, 2, 2, 2, 2, 2, 2, 2], 0, 0, 2048, 2048),
    ([0, 0, 0, 0], 0, 9, 256, 256),
    ([5, 40, 0, 17, 33], 4, 3, 500, 640),
    ([64, 1, 63, 65], 0, 1, 384, 1152),
    ([200, 0, 130, 1, 128, 129, 300], 2, 50, 1000, 520),
    ([700, 5, 256, 257], 0, 0, 640, 3584),
    ([1] * 100 + [0] * 27 + [50], 0, 0, 260, 384),
    ([3] * 1024, 0, 0, 40, 136),
    ([0] * 63 + [1500], 1, 1, 512, 256),
]


@pytest.mark.parametrize("counts,front,behind,N,K", GROUPED, ids=lambda v: str(v)[:24])
def test_grouped(hxq, counts, front, behind, N, K):
    import torch
    E, M = len(counts), front + sum(counts) + behind
    xq, xs = make_activation(M + N, M, K)
    wq, ws = make_weights(N + K, E, N, K)
    bias = randn(78, E, N)
    off = offsets_of(counts, front)
    lin = hxq.Fp8Linear(wq, ws)
    for out, b in ((hxq.HXQ_OUT_F32, None), (hxq.HXQ_OUT_BF16, bias)):
        dt = torch.bfloat16 if out == hxq.HXQ_OUT_BF16 else torch.float32
        y = torch.full((M, N), 7.0, dtype=dt, device="cuda")
        lin.forward_grouped(xq, xs, off, bias=b, out_dtype=out, y=y)
        at = front
        for e, n in enumerate(counts):
            if n:
                check_product(y[at:at + n], dense_x(xq[at:at + n], xs[at:at + n], K), dense_w(wq[e], ws[e]),
                              b[e] if b is not None else None, f"expert {e}, {n} rows")
            at += n
        assert (y[:front] == 7).all() and (y[M - behind:] == 7).all(), "rows of no expert were written"
    lin.check()


def test_grouped_with_one_expert_is_the_layer(hxq):
    import torch
    wq, ws = make_weights(3, 1, 500, 700)
    for M in (1, 50, 400):
        xq, xs = make_activation(4, M, 700)
        a = hxq.Fp8Linear(wq[0], ws[0]).forward(xq, xs)
        b = hxq.Fp8Linear(wq, ws).forward_grouped(xq, xs, offsets_of([M]))
        assert torch.equal(a, b)


@pytest.mark.parametrize("M", [12, 600])
def test_grouped_survives_bad_offsets(hxq, M):
    """Offsets that fall or leave [0, M] are clamped: nothing outside y is written, and the handle works afterwards."""
    import torch
    E, N, K = 4, 200, 256
    xq, xs = make_activation(1, M, K)
    wq, ws = make_weights(2, E, N, K)
    lin = hxq.Fp8Linear(wq, ws)
    good = offsets_of([M // 4] * 4)
    want = lin.forward_grouped(xq, xs, good)
    for bad in ([5, 2, 9, 1, 4], [-7, -3, 2, 10**9, 3], [2**31 - 1] * 5, [-2**31] * 5, [0, M, 0, M, 2 * M]):
        buf = torch.full((M + 2, N), 7.0, device="cuda")
        lin.forward_grouped(xq, xs, torch.tensor(bad, dtype=torch.int32, device="cuda"), y=buf[1:M + 1])
        torch.cuda.synchronize()
        assert (buf[0] == 7).all() and (buf[-1] == 7).all()
    assert torch.equal(lin.forward_grouped(xq, xs, good), want)
    lin.check()


# ---- sizes past 32 bits ------------------------------------------------------------

def test_more_than_2_31_outputs(hxq):
    """y of 2.2e9 elements: rows at both ends and around element 2^31."""
    import torch
    M, N, K = 55000, 40016, 144
    xq, xs = make_activation(1, M, K)
    wq, ws = make_weights(2, 1, N, K)
    y = hxq.Fp8Linear(wq[0], ws[0]).forward(xq, xs, out_dtype=hxq.HXQ_OUT_BF16)
    w = dense_w(wq[0], ws[0])
    mid = 2**31 // N
    for r in (slice(0, 40), slice(mid - 20, mid + 20), slice(M - 40, M)):
        check_product(y[r], dense_x(xq[r], xs[r], K), w, None, f"rows {r}")


def test_more_than_2_31_weights(hxq):
    """Experts whose weights take 2.3 GB: the first and the last, few rows and many."""
    import torch
    E, N, K = 34, 8200, 8208
    wq = torch.empty(E, N, K, dtype=torch.float8_e4m3fn, device="cuda")
    for e in range(E):
        wq[e] = randn(e, N, K, scale=100.0).clamp_(-448, 448).to(torch.float8_e4m3fn)
    ws = 3e-4 * torch.exp(randn(99, E, 65, 65))
    lin = hxq.Fp8Linear(wq, ws)
    for n in (3, 300):
        xq, xs = make_activation(5, 2 * n, K)
        y = lin.forward_grouped(xq, xs, offsets_of([n] + [0] * (E - 2) + [n]))
        for e, r in ((0, slice(0, n)), (E - 1, slice(n, 2 * n))):
            check_product(y[r], dense_x(xq[r], xs[r], K), dense_w(wq[e], ws[e]), None, f"expert {e}")


def test_more_than_2_31_elements_quantized(hxq):
    import torch
    M, K = 70001, 32000
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda").normal_()
    mid = 2**31 // K
    rows = [0, 1, mid - 1, mid, mid + 1, M - 1]
    q, s = hxq.fp8_quantize(x)
    check_bytes(q[rows], s[rows], f64(x[rows]), K)
    del q, s
    x = x.view(-1)[:2**31 + 2**20].view(-1, 16384)  # 131136 rows
    q, s, _, _ = hxq.rmsnorm(x)
    rows = [0, 131071, 131072, x.shape[0] - 1]
    check_bytes(q[rows], s[rows], ref_norm(x[rows], None, None, 1e-6)[1], 16384, DELTA)


# ---- streams, graphs, refusals -----------------------------------------------------------

def test_zero_rows(hxq):
    import torch
    wq, ws = make_weights(3, 1, 130, 200)
    q, s = hxq.fp8_quantize(torch.zeros(0, 200, device="cuda"))
    assert q.shape == (0, 208) and s.shape == (0, 2)
    assert hxq.Fp8Linear(wq[0], ws[0]).forward(q, s).shape == (0, 130)
    assert hxq.Fp8Linear(wq, ws).forward_grouped(q, s, offsets_of([0])).shape == (0, 130)
    assert hxq.rmsnorm(torch.zeros(0, 200, device="cuda"), want="y")[2].shape == (0, 200)
    assert hxq.fp8_swiglu(torch.zeros(0, 400, device="cuda"))[0].shape == (0, 208)


def test_two_streams_on_one_handle(hxq):
    """Calls of one handle that overlap on two streams: there is no workspace to share."""
    import torch
    wq, ws = make_weights(3, 1, 2048, 2048)
    lin = hxq.Fp8Linear(wq[0], ws[0])
    xs_ = [make_activation(i, m, 2048) for i, m in enumerate((1, 8, 60, 300))]
    want = [lin.forward(*x) for x in xs_]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[torch.empty_like(w) for w in want] for _ in streams]
    for _ in range(20):
        for st, ys in zip(streams, got):
            for x, y in zip(xs_, ys):
                lin.forward(*x, y=y, stream=st)
    torch.cuda.synchronize()
    for ys in got:
        assert all(torch.equal(a, b) for a, b in zip(ys, want))
    lin.check()


def test_two_graphs_of_one_handle_at_once(hxq):
    """Graphs captured from the same handles, replayed over one another on two streams."""
    import torch
    wq, ws = make_weights(3, 4, 1024, 1152)
    lin, ex = hxq.Fp8Linear(wq[0], ws[0]), hxq.Fp8Linear(wq, ws)
    graphs = []
    for i, m in enumerate((5, 40)):
        q, s = make_activation(i, m, 1152)
        Q, S = make_activation(10 + i, 20 * m, 1152)
        off = offsets_of([3 * m, 0, 16 * m, m])
        want = [lin.forward(q, s), lin.forward(Q, S), ex.forward_grouped(Q, S, off)]
        st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=st):
            got = [lin.forward(q, s), lin.forward(Q, S), ex.forward_grouped(Q, S, off)]
        graphs.append((g, st, want, got, (q, s, Q, S, off)))  # (the graph's inputs stay alive)
    torch.cuda.synchronize()
    for _ in range(30):
        for g, st, *_ in graphs:
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for _, _, want, got, _ in graphs:
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    ex.check()


def test_host_threads(hxq):
    """Calls from several host threads, each on a stream of its own."""
    import threading
    import torch
    wq, ws = make_weights(3, 1, 640, 512)
    lin = hxq.Fp8Linear(wq[0], ws[0])
    x = randn(1, 70, 512)
    want = lin.forward(*hxq.fp8_quantize(x))
    torch.cuda.synchronize()
    bad = []

    def work():
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                for _ in range(50):
                    y = lin.forward(*hxq.fp8_quantize(x))
                st.synchronize()
            if not torch.equal(y, want):
                bad.append("differs")
        except Exception as e:  # noqa: BLE001
            bad.append(repr(e))

    ts = [threading.Thread(target=work) for _ in range(4)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not bad, bad


def mlp(hxq, x, res, w, gate_up, down, bufs):
    """norm -> gate|up -> gated activation -> down, every output in a buffer of its own."""
    q, s, _, t = hxq.rmsnorm(x, w, 1e-6, residual=res, sum_out=bufs["sum"], q=bufs["q"], scales=bufs["s"])
    gu = gate_up.forward(q, s, out_dtype=hxq.HXQ_OUT_BF16, y=bufs["gu"])
    q2, s2 = hxq.fp8_swiglu(gu, q=bufs["q2"], scales=bufs["s2"])
    return down.forward(q2, s2, out_dtype=hxq.HXQ_OUT_BF16, y=bufs["y"]), t


def mlp_buffers(M, K, H):
    import torch
    e = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    f8 = torch.float8_e4m3fn
    return {"sum": e(M, K), "q": e(M, -(-K // 16) * 16, dt=f8), "s": e(M, -(-K // 128), dt=torch.float32),
            "gu": e(M, 2 * H), "q2": e(M, -(-H // 16) * 16, dt=f8), "s2": e(M, -(-H // 128), dt=torch.float32),
            "y": e(M, K)}


@pytest.mark.parametrize("M", [1, 24, 300])
def test_mlp_block(hxq, M):
    """The operators as they are used together, eager and as a captured graph replayed on new inputs, against the
    float64 block on unquantised weights. Each 8-bit tensor has relative errors below 2^-4, in rms below
    2^-4 / sqrt(3) = 0.037; four of them in a row, and errors of the gate that its product passes on at most
    doubled, stay below sqrt(4) * 2 * 0.037 = 0.15 of the result's norm."""
    import torch
    K, H = 1024, 2816
    x, res = randn(1, M, K).bfloat16(), randn(2, M, K, scale=3.0).bfloat16()
    w = 1 + randn(3, K, scale=0.1)
    Wgu, Wd = randn(4, 2 * H, K, scale=K ** -0.5), randn(5, K, H, scale=H ** -0.5)
    gate_up, down = hxq.Fp8Linear.from_weight(Wgu), hxq.Fp8Linear.from_weight(Wd.bfloat16())
    bufs = mlp_buffers(M, K, H)

    def want():
        t, h = ref_norm(x, res, w, 1e-6)
        gu = torch.tensor(h, device="cuda") @ Wgu.double().t()
        g, u = gu[:, :H], gu[:, H:]
        return (g / (1 + torch.exp(-g)) * u) @ Wd.double().t(), t

    def check(got):
        ref, t = want()
        assert torch.equal(got[1], t)
        assert float((got[0].double() - ref).norm() / ref.norm()) < 0.15

    check(mlp(hxq, x, res, w, gate_up, down, bufs))
    eager = bufs["y"].clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        mlp(hxq, x, res, w, gate_up, down, bufs)
        with torch.cuda.graph(graph, stream=st):
            got = mlp(hxq, x, res, w, gate_up, down, bufs)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(bufs["y"], eager)
    x.copy_(randn(11, M, K).bfloat16())
    res.copy_(randn(12, M, K).bfloat16())
    graph.replay()
    torch.cuda.synchronize()
    check(got)
    gate_up.check()
    down.check()


def test_experts_block(hxq):
    """Tokens to their two experts and back: grouped gate|up, gated activation, grouped down, weighted sum; each
    step's operator against its formula on the bytes that it was given."""
    import torch
    T, E, K, H = 37, 6, 512, 640
    x = randn(1, T, K).bfloat16()
    Wgu, Wd = randn(2, E, 2 * H, K, scale=K ** -0.5), randn(3, E, K, H, scale=H ** -0.5)
    gate_up, down = hxq.Fp8Linear.from_weight(Wgu), hxq.Fp8Linear.from_weight(Wd)
    prob, expert = torch.softmax(randn(4, T, E), 1).topk(2, dim=1)
    flat = expert.reshape(-1)
    order = torch.argsort(flat, stable=True)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = torch.cumsum(torch.bincount(flat, minlength=E), 0)
    q, s = hxq.fp8_quantize(x)
    rows = order // 2
    q, s = codes_t(q)[rows].contiguous(), s[rows].contiguous()
    gu = gate_up.forward_grouped(q, s, off, out_dtype=hxq.HXQ_OUT_BF16)
    q2, s2 = hxq.fp8_swiglu(gu)
    y = down.forward_grouped(q2, s2, off)
    wq, ws = hxq.fp8_encode(Wgu)
    wq2, ws2 = hxq.fp8_encode(Wd)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        check_product(gu[a:b], dense_x(q.view(torch.float8_e4m3fn)[a:b], s[a:b], K), dense_w(wq[e], ws[e]), None)
        check_product(y[a:b], dense_x(q2[a:b], s2[a:b], H), dense_w(wq2[e], ws2[e]), None)
    out = torch.zeros(T, K, device="cuda").index_add_(0, rows, y * prob.reshape(-1)[order][:, None])
    X = x.double()
    ref = torch.zeros(T, K, dtype=torch.float64, device="cuda")
    for e in range(E):
        g, u = (X @ Wgu[e].double().t()).chunk(2, 1)
        ye = (g / (1 + torch.exp(-g)) * u) @ Wd[e].double().t()
        ref += ye * (prob.double() * (expert == e)).sum(1, keepdim=True)
    assert float((out.double() - ref).norm() / ref.norm()) < 0.15  # as test_mlp_block


def test_norm_feeds_a_codebook_layer_and_its_weights_transcode(hxq):
    """rmsnorm's bf16 output into HelixLinear, and that layer's decoded weights as an 8-bit layer."""
    import torch
    import synthetic
    layer = synthetic.make_layer(0, 512, 640, 5, sidecar_count=200)
    lin = hxq.HelixLinear.from_layer(layer)
    W = lin.decode()
    x = randn(1, 40, 640)
    _, _, y, _ = hxq.rmsnorm(x, want="y")
    got = lin.forward_out(y)
    ref = y.double() @ W.double().t()
    assert ((got.double() - ref).abs() <= 8e-3 * (y.double().abs() @ W.double().abs().t())).all()
    q, s, _, _ = hxq.rmsnorm(x)
    got8 = hxq.Fp8Linear.from_weight(W).forward(q, s)
    assert float((got8.double() - ref).norm() / ref.norm()) < 0.1  # two 8-bit tensors: sqrt(2) * 0.037, doubled


def test_handle_refusals(hxq):
    import torch
    wq, ws = make_weights(1, 2, 64, 96)
    two, one = hxq.Fp8Linear(wq, ws), hxq.Fp8Linear(wq[0], ws[0])
    xq, xs = make_activation(2, 4, 96)
    y = torch.empty(4, 64, device="cuda")
    p = lambda t: t.data_ptr()  # noqa: E731
    f, g, E = hxq.lib.hxq_fp8_forward, hxq.lib.hxq_fp8_forward_grouped, hxq.HXQ_EINVAL
    assert f(two.handle, p(xq), p(xs), None, p(y), 0, 4, None) == E
    assert f(one.handle, None, p(xs), None, p(y), 0, 4, None) == E
    assert f(one.handle, p(xq), None, None, p(y), 0, 4, None) == E
    assert f(one.handle, p(xq), p(xs), None, None, 0, 4, None) == E
    assert f(one.handle, p(xq), p(xs), None, p(y), 2, 4, None) == E
    assert f(one.handle, p(xq), p(xs), None, p(y), 0, -1, None) == E
    assert f(one.handle, p(xq) + 8, p(xs), None, p(y), 0, 3, None) == E
    assert f(one.handle, p(xq), p(xs), None, p(y) + 2, 0, 3, None) == E
    assert f(one.handle, p(xq), p(xs), None, p(y), 0, 2**31 - 1, None) == E
    assert g(two.handle, p(xq), p(xs), None, None, p(y), 0, 4, None) == E
    host = np.zeros(256, np.uint8)
    x = torch.zeros(4, 32, device="cuda")
    assert hxq.lib.hxq_fp8_quantize(p(x), 0, 1, 32, (host.ctypes.data + 15) // 16 * 16, p(xs), None) == E  # pageable
    assert hxq.hxq_fp8_info(two.handle) == (2, 64, 96)
    for call in (lambda: one.forward(xq[:, :80], xs), lambda: one.forward(xq, xs[:2]), lambda: one.forward(xq, xs.double()),
                 lambda: one.forward(xq, xs, bias=torch.zeros(63, device="cuda")),
                 lambda: one.forward(xq, xs, y=y.bfloat16()), lambda: one.forward(xq, xs, y=y.t()),
                 lambda: two.forward(xq, xs), lambda: one.forward_grouped(xq, xs, offsets_of([4])),
                 lambda: two.forward_grouped(xq, xs, offsets_of([4])),
                 lambda: two.forward_grouped(xq, xs, offsets_of([2, 2]).long()),
                 lambda: two.forward_grouped(xq, xs, offsets_of([2, 2]).cpu()),
                 lambda: hxq.fp8_swiglu(torch.zeros(2, 31, device="cuda")),
                 lambda: hxq.fp8_quantize(torch.zeros(2, 32, device="cuda", dtype=torch.float16)),
                 lambda: hxq.rmsnorm(x, residual=x[:2]), lambda: hxq.rmsnorm(x, sum_out=x),
                 lambda: one.forward(xq.cpu(), xs.cpu(), y=y.cpu()), lambda: one.forward(xq, xs.cpu()),
                 lambda: one.forward(xq, xs, y=y.cpu()), lambda: hxq.rmsnorm(x, scales=xs, want="y"),
                 lambda: hxq.rmsnorm(x, torch.ones(31, device="cuda")), lambda: hxq.rmsnorm(x, want="z")):
        with pytest.raises(hxq.HXQError) as e:
            call()
        assert e.value.code == hxq.HXQ_EINVAL
