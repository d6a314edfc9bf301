"""The 8-bit-float kernels beyond their first pieces: persistent loops that come round, rings that are filled
again, pieces and pairs that end early. Forms and tolerances are those of test_gpu_fp8."""
import pytest

from test_gpu_fp8 import (DELTA, check_bytes, check_product, check_y, codes, dense_w, dense_x, dtype, make_activation,
                          make_weights, offsets_of, randn, ref_norm, unaligned)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out", [0, 1])
def test_pairs_with_one_empty_half(hxq, out):
    """Blocks of 256 tokens of which at most 128 exist: the second CTA of a pair stores nothing and comes to the end
    with its last arrivals in the first one just sent. Launches follow one another at once; every one gives the same
    bits, and no wait runs out."""
    import torch
    E, N, K, n = 40, 1024, 512, 120
    xq, xs = make_activation(1, E * n, K)
    wq, ws = make_weights(2, E, N, K)
    off = offsets_of([n] * E)
    lin = hxq.Fp8Linear(wq, ws)
    ys = [lin.forward_grouped(xq, xs, off, out_dtype=out) for _ in range(60)]
    one = hxq.Fp8Linear(wq[0], ws[0])
    zs = [one.forward(xq[:1400], xs[:1400], out_dtype=out) for _ in range(60)]  # (5 blocks and 120 rows)
    lin.check()
    one.check()
    assert all(torch.equal(y, ys[0]) for y in ys) and all(torch.equal(z, zs[0]) for z in zs)
    for e in range(E):
        r = slice(e * n, (e + 1) * n)
        check_product(ys[0][r], dense_x(xq[r], xs[r], K), dense_w(wq[e], ws[e]), None, f"expert {e}")
    check_product(zs[0], dense_x(xq[:1400], xs[:1400], K), dense_w(wq[0], ws[0]), None)


# (M, N, K, rows per expert or None): each kernel, one CTA and clusters and pairs, and the experts' forms
WITHHELD = [(1, 11008, 1024, None), (29, 2048, 4096, None), (60, 2048, 4096, None), (512, 2048, 2048, None),
            (16, 1024, 2048, [3, 0, 9, 4]), (200, 512, 2048, [50] * 4), (4800, 1024, 512, [120] * 40)]


@pytest.mark.parametrize("M,N,K,counts", WITHHELD, ids=lambda v: str(v)[:12])
@pytest.mark.parametrize("stage", [0, 1])
def test_withheld_activations_time_out_then_recover(hxq, M, N, K, counts, stage):
    """Each CTA's stage never gets its activations: the waits run out (1 ms), the CTAs let go of what they hold and
    return, check reports it once, and the next products on the handle are right."""
    import torch
    xq, xs = make_activation(1, M, K)
    wq, ws = make_weights(2, len(counts or [1]), N, K)
    lin = hxq.Fp8Linear(wq, ws) if counts else hxq.Fp8Linear(wq[0], ws[0])
    off = offsets_of(counts) if counts else None
    run = (lambda: lin.forward_grouped(xq, xs, off)) if counts else (lambda: lin.forward(xq, xs))
    want = run()
    check_product(want[:1], dense_x(xq[:1], xs[:1], K), dense_w(wq[0], ws[0]), None)
    lin.check()
    y = torch.empty_like(want)
    hxq.hxq_test_fp8_forward_withheld(lin.handle, xq, xs, off, y, M, -1, 100000)
    torch.cuda.synchronize()
    lin.check()
    assert torch.equal(y, want)  # nothing withheld: the product
    hxq.hxq_test_fp8_forward_withheld(lin.handle, xq, xs, off, y, M, stage, 1000)
    torch.cuda.synchronize()
    assert hxq.lib.hxq_fp8_check(lin.handle) == hxq.HXQ_ETIMEOUT
    assert hxq.lib.hxq_fp8_check(lin.handle) == hxq.HXQ_OK  # reported once, then cleared
    for _ in range(3):
        assert torch.equal(run(), want)
    lin.check()


@pytest.mark.parametrize("M,N,K", [(1, 1024, 512), (20, 256, 2048), (512, 2048, 2048)])
def test_waits_do_not_count_the_previous_kernel(hxq, M, N, K):
    """A product launched early behind a kernel that releases its dependents at once and then runs for longer than the
    product's waits may take: it waits for that kernel's end first, and then runs."""
    import torch
    xq, xs = make_activation(1, M, K)
    wq, ws = make_weights(2, 1, N, K)
    lin = hxq.Fp8Linear(wq[0], ws[0])
    want = lin.forward(xq, xs)
    # two rows of 2^25 columns: two CTAs, some milliseconds, and nearly every SM free for the product
    x = torch.ones(2, 2**25, device="cuda")
    y = torch.empty(2, 2**25, dtype=torch.bfloat16, device="cuda")
    hxq.rmsnorm(x, y=y)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    hxq.rmsnorm(x, y=y)
    b.record()
    torch.cuda.synchronize()
    limit = int(a.elapsed_time(b) * 1000 / 4)
    assert limit > 200, "the kernel in front is too short for this test"
    got = torch.empty_like(want)
    hxq.rmsnorm(x, y=y)
    hxq.hxq_test_fp8_forward_withheld(lin.handle, xq, xs, None, got, M, -1, limit)
    torch.cuda.synchronize()
    lin.check()
    assert torch.equal(got, want)


@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("K", [8, 250, 3000, 10008, 33000])
def test_rmsnorm_padding_is_zero_whatever_the_root(hxq, xt, K):
    """Bytes past K are 0 in rows whose root is NaN, infinite (zeros without eps) or 0, too."""
    x = randn(K, 5, K)
    x[1, 3] = float("nan")
    x[2, 4] = float("inf")
    x[3] = 0
    x = x.to(dtype(xt))
    for t in (x, unaligned(x)):
        for eps in (0.0, 1e-6):
            q, s, y, _ = hxq.rmsnorm(t, None, eps, want="qy")
            assert codes(q).shape[1] > K and not codes(q)[:, K:].any()
            _, h = ref_norm(x, None, None, eps)
            check_bytes(q[[0, 4]], s[[0, 4]], h[[0, 4]], K, DELTA)
            assert ((codes(q)[1, :K] & 0x7F) == 0x7F).all()
            check_y(y[[0, 3, 4]], h[[0, 3, 4]])


@pytest.mark.parametrize("xt,rt", [("f32", None), ("bf16", None), ("f32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("K", [256, 250, 3000, 10000, 33000])
def test_rmsnorm_rows_of_subnormals_without_eps(hxq, xt, rt, K):
    """1 / root beyond fp32's end: y and the 8 bits are ordinary all the same, zeros stay zeros, and a large weight
    or one of 0 changes nothing of that. Rows of zeros are 0 / 0."""
    import torch
    x = randn(K, 7, K)
    x[0] *= 1e-40
    x[1] *= 1e-42
    x[2, 1:] = 0
    x[2, 0] = 2.0 ** -130
    x[3] *= 1e-40
    x[3, :128] = 0
    x[4] *= 1e-38  # (just inside)
    x[5] = 0
    x = x.to(dtype(xt))
    res = None
    if rt:  # t = x + residual is x, with its signs as they are
        res = torch.zeros(7, K, device="cuda", dtype=dtype(rt))
    for big in (1.0, 2.0 ** 60):
        w = (1 + randn(K + 1, K, scale=0.2)) * big
        w[7], w[200] = 0, 0
        t, h = ref_norm(x, res, w, 0.0)
        for copy in (lambda v: v, unaligned):
            q, s, y, total = hxq.rmsnorm(copy(x), w, 0.0, residual=res, want="qy")
            _, _, y1, _ = hxq.rmsnorm(copy(x), w, 0.0, residual=res, want="y")
            if res is not None:
                assert torch.equal(total, t)
            check_bytes(q, s, h, K, DELTA)
            check_y(y, h)
            assert torch.equal(y1.view(torch.int16), y.view(torch.int16))


@pytest.mark.parametrize("out", ["y", "q", "scales", "sum"])
def test_rmsnorm_refuses_each_output_in_pageable_memory(hxq, out):
    """Outputs that the GPU cannot reach are refused on the host, whichever they are."""
    import numpy as np
    import torch
    x, res = randn(1, 2, 32), randn(2, 2, 32)
    host = np.zeros(1024, np.uint8)
    p = {"y": torch.empty(2, 32, dtype=torch.bfloat16, device="cuda"), "q": torch.empty(2, 32, dtype=torch.uint8, device="cuda"),
         "scales": torch.empty(2, 1, device="cuda"), "sum": torch.empty(2, 32, device="cuda")}
    at = {k: v.data_ptr() for k, v in p.items()}
    at[out] = (host.ctypes.data + 15) // 16 * 16
    rc = hxq.lib.hxq_rmsnorm(x.data_ptr(), 0, res.data_ptr(), at["sum"], 0, None, 1e-6, 2, 32, at["y"], at["q"],
                             at["scales"], None)
    assert rc == hxq.HXQ_EINVAL


# ---- persistent loops, rings, clusters with more than one unit --------------------------

NORM_LOOPS = [
    # (rows, K): several rows for each resident CTA at each depth of the ring and number of pieces
    (9001, 200), (5003, 2048), (4001, 3592), (3001, 10000), (2003, 16384), (4099, 1000),
]


@pytest.mark.parametrize("xt,rt", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", None),
                                   ("bf16", None)])
@pytest.mark.parametrize("M,K", NORM_LOOPS)
def test_rmsnorm_rows_one_after_another(hxq, M, K, xt, rt):
    """CTAs that take many rows: each row against float64, with the sum in place of the residual. A few rows among
    them need their mean in 64 bits (from shared memory, while later rows arrive), are zeros, or hold a NaN."""
    import torch
    x = randn(M + K, M, K).to(dtype(xt))
    x[5::611] *= 1e25
    x[11::613] *= 1e-30
    x[17::617] = 0
    x[23::619, K // 2] = float("nan")
    res = randn(M + K + 1, M, K, scale=2.0).to(dtype(rt)) if rt else None
    if rt:
        res[5::611] *= 1e25
        res[11::613] *= 1e-30
        res[17::617] = 0
    w = 1 + randn(M + K + 2, K, scale=0.2)
    t = x if res is None else (x.float() + res.float()).to(res.dtype)
    own = res.clone() if rt else None
    q, s, y, total = hxq.rmsnorm(x, w, 1e-6, residual=own, sum_out=own, want="qy")
    if rt:
        assert torch.equal(total.nan_to_num(7.0), t.nan_to_num(7.0)) and torch.equal(total.isnan(), t.isnan())
    d = t.double()
    h = d / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-6) * w.double()
    # y of every row, on the GPU
    ok = (y.double() - h).abs() <= (2.0 ** -8 + DELTA) * h.abs() + 2.0 ** -133
    assert (ok | (h.isnan() & y.isnan())).all()
    # scales of every block: the smallest power of two with max <= 448 s
    kb = -(-K // 128)
    a = torch.zeros(M, kb * 128, dtype=torch.float64, device="cuda")
    a[:, :K] = h.abs().nan_to_num(0.0)
    a = a.view(M, kb, 128).amax(2)
    m, e = torch.frexp(a / 448)
    want = torch.where(a == 0, 1.0, torch.ldexp(torch.ones_like(m), (e - (m == 0.5).int()).clamp(-126, 120)))
    assert torch.equal(s.double(), want)
    # every byte within the rounding of h to e4m3: half a step of 2^-3 of its binade, 2^-10 at the least
    v = h / want.repeat_interleave(128, 1)[:, :K]
    got = q[:, :K].double()
    step = torch.ldexp(torch.ones_like(v), (torch.frexp(v.abs().nan_to_num(1.0))[1] - 1).clamp(min=-6) - 3)
    assert ((got - v).abs() <= step / 2 + DELTA * v.abs()).logical_or(v.isnan() & got.isnan()).all()
    assert not q.view(torch.uint8)[:, K:].any()
    # and some rows byte by byte, the special ones and the last ones among them
    rows = [0, 1, 5, 11, 17, 5 + 611, 11 + 613, 17 + 617, M // 2, M - 2, M - 1]
    check_bytes(q[rows], s[rows], h[rows].cpu().numpy(), K, DELTA)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("E,N,K", [(1, 6000, 4000), (3, 1500, 4104), (1, 128, 131072), (1, 6000, 1001)])
def test_encode_blocks_one_after_another(hxq, E, N, K, dt):
    """Five and more blocks for each SM: slots that are filled again. Every byte against float64, with blocks of
    zeros, NaN, infinities and numbers below fp32's normal ones among them."""
    import torch
    W = randn(N + K, E, N, K, scale=0.02)
    W *= torch.exp2(torch.randint(-20, 20, (E, -(-N // 128), -(-K // 128)), device="cuda").float()) \
        .repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    W[0, 0, 130] = float("nan")
    W[0, -1, -1] = float("inf")
    W[-1, 50, 300] = -float("inf")
    W[0, :128, 384:512] = 0
    W[0, :128, 512:640] = W[0, :128, 512:640].sign() * 1e-41
    W = W.to(dtype(dt))
    q, s = hxq.fp8_encode(W)
    for e in range(E):
        nb, kb = -(-N // 128), -(-K // 128)
        a = torch.zeros(nb * 128, kb * 128, dtype=torch.float64, device="cuda")
        a[:N, :K] = W[e].double().abs().nan_to_num(0.0, posinf=3.402823466e38)
        a = a.view(nb, 128, kb, 128).amax((1, 3))
        m, x = torch.frexp(a / 448)
        want = torch.where(a == 0, 1.0, torch.ldexp(torch.ones_like(m), (x - (m == 0.5).int()).clamp(-126, 120)))
        assert torch.equal(s[e].double(), want)
        full = want.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
        v = W[e].double() / full
        v[v.isinf()] = float("nan")
        # torch rounds fp32 to e4m3 to nearest even; v is exact in fp32 unless below its normal numbers, where both are 0
        ref = v.float().to(torch.float8_e4m3fn).float()
        got = q[e].float()
        assert torch.equal(got.nan_to_num(999.0), ref.nan_to_num(999.0)) and torch.equal(got.isnan(), ref.isnan())


@pytest.mark.parametrize("counts,N,K", [([2] * 8, 2048, 14336), ([0, 5, 1, 0, 7, 1, 1, 1], 2048, 14336),
                                        ([20] * 8, 1024, 8192), ([40] * 4, 2048, 8192), ([60, 3, 64, 50], 1500, 8200)],
                         ids=lambda v: str(v)[:20])
@pytest.mark.parametrize("out", [0, 1])
def test_clusters_with_several_units(hxq, counts, N, K, out):
    """Clusters that exchange sums for one unit after another: the receiving rows are used again."""
    import torch
    E, M = len(counts), sum(counts)
    xq, xs = make_activation(M, M, K)
    wq, ws = make_weights(N, E, N, K)
    lin = hxq.Fp8Linear(wq, ws)
    y = lin.forward_grouped(xq, xs, offsets_of(counts), out_dtype=out)
    at = 0
    for e, n in enumerate(counts):
        if n:
            check_product(y[at:at + n], dense_x(xq[at:at + n], xs[at:at + n], K), dense_w(wq[e], ws[e]), None, f"expert {e}")
        at += n
    for _ in range(5):
        assert torch.equal(lin.forward_grouped(xq, xs, offsets_of(counts), out_dtype=out), y)
    lin.check()


@pytest.mark.parametrize("M", [16, 30, 64])
@pytest.mark.parametrize("out", [0, 1])
def test_clusters_with_two_units_of_one_layer(hxq, M, out):
    """86 tiles for some 45 clusters of three."""
    import torch
    N, K = 11008, 8192
    xq, xs = make_activation(M, M, K)
    wq, ws = make_weights(N, 1, N, K)
    bias = randn(4, N)
    lin = hxq.Fp8Linear(wq[0], ws[0])
    y = lin.forward(xq, xs, bias=bias, out_dtype=out)
    check_product(y, dense_x(xq, xs, K), dense_w(wq[0], ws[0]), bias)
    for _ in range(5):
        assert torch.equal(lin.forward(xq, xs, bias=bias, out_dtype=out), y)
    lin.check()


# (512 x 2048 x 2048: 16 units on 74 pairs, pieces of 64 features; 1100 x 2048: 40, pieces of 128)
@pytest.mark.parametrize("M,N,K", [(512, 2048, 2048), (512, 1920, 2048), (300, 2048, 2048), (512, 2008, 2048),
                                   (1100, 2048, 2048), (290, 2177, 2048), (512, 2500, 2048)])
def test_units_cut_into_pieces(hxq, M, N, K):
    """The last round's units by pieces of 64 or 128 features: stores narrower than a box of 128 bytes, odd tiles and
    ends of rows among them."""
    import torch
    xq, xs = make_activation(M, M, K)
    wq, ws = make_weights(N, 1, N, K)
    bias = randn(3, N)
    lin = hxq.Fp8Linear(wq[0], ws[0])
    x, w = dense_x(xq, xs, K), dense_w(wq[0], ws[0])
    for out in (hxq.HXQ_OUT_F32, hxq.HXQ_OUT_BF16):
        for b in (None, bias):
            buf = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16 if out else torch.float32, device="cuda")
            y = lin.forward(xq, xs, bias=b, out_dtype=out, y=buf[1:M + 1])
            check_product(y, x, w, b, f"out={out}")
            assert (buf[0] == 7).all() and (buf[-1] == 7).all()
    lin.check()


FIRST_CALLS_CAPTURED = """
import torch
import vq_compressed_linear_b200 as hxq
W, W2 = torch.randn(640, 512, device="cuda"), torch.randn(2, 640, 512, device="cuda")
w, off = torch.ones(512, device="cuda"), torch.tensor([0, 1, 1], dtype=torch.int32, device="cuda")
lin, ex = hxq.Fp8Linear(*hxq.fp8_encode(W)), hxq.Fp8Linear(*hxq.fp8_encode(W2))
xs = [torch.randn(m, 512, device="cuda").bfloat16() for m in (1, 20, 60, 600)]

def run():
    out = []
    for x in xs:
        q, s, y, t = hxq.rmsnorm(x, w, 1e-6, residual=x, want="qy")
        out += [lin(q, s), y, t, lin(*hxq.fp8_quantize(x)), lin(*hxq.fp8_swiglu(torch.cat([x, x], 1)))]
        y = torch.zeros(x.shape[0], 640, device="cuda")
        out.append(ex.forward_grouped(*hxq.fp8_quantize(x.float()), off, y=y))
    return out

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
graph.replay()
torch.cuda.synchronize()
lin.check()
ex.check()
assert all(torch.equal(a, b) for a, b in zip(got, run()))
print("equal")
"""


def test_first_calls_of_a_process_captured():
    """What a call looks up or sets once (kernel attributes, residency) is no harm to a capture that it falls into."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS_CAPTURED], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "equal", r.stderr[-2000:]


def test_longest_rows(hxq):
    """One row of 2^31 - 1 columns through the norm, the quantiser and the encoder: both ends and the middle."""
    import torch
    K = 2**31 - 1
    x = torch.empty(1, K, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    x[0, K - 128:] *= 1000  # (the last block's scale is its own)
    ss = sum(x[0, i:i + 2**27].double().square().sum() for i in range(0, K, 2**27))
    parts = [slice(0, 1024), slice(2**30, 2**30 + 1024), slice(K // 128 * 128 - 1024, K)]

    def check(q, s, f, delta):
        for p in parts:
            h = f(x[:, p].double())
            n = h.shape[1]
            at = slice(p.start // 128, p.start // 128 + -(-n // 128))
            check_bytes(q[:, p.start:p.start + -(-n // 16) * 16], s[:, at], h.cpu().numpy(), n, delta)

    q, s = hxq.fp8_quantize(x)
    assert q.shape == (1, 2**31) and codes(q[:, -16:])[0, 15] == 0
    check(q, s, lambda v: v, 0.0)
    q, s, y, _ = hxq.rmsnorm(x, None, 0.0, want="qy")
    root = torch.sqrt(ss / K)
    check(q, s, lambda v: v / root, DELTA)
    for p in parts:
        check_y(y[:, p], (x[:, p].double() / root).cpu().numpy())
    del q, s, y
    q, s = hxq.fp8_encode(x)
    for p in parts:
        n = min(p.stop, K) - p.start
        at = slice(p.start // 128, p.start // 128 + -(-n // 128))
        check_bytes(q[:, p], s[:, at], x[:, p].double().cpu().numpy(), n, rows=128)


# ---- forms that the documentation allows ------------------------------------------------

@pytest.mark.parametrize("K", [250, 2048, 5000, 33000])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_rmsnorm_sum_in_place_of_x(hxq, dt, K):
    """sum may be x; x and the residual may be one tensor."""
    import torch
    x, res = randn(1, 700, K).to(dtype(dt)), randn(2, 700, K).to(dtype(dt))
    q, s, y, t = hxq.rmsnorm(x, None, 1e-6, residual=res, want="qy")
    own = x.clone()
    q1, s1, y1, t1 = hxq.rmsnorm(own, None, 1e-6, residual=res, sum_out=own, want="qy")
    assert t1 is own and torch.equal(own, t) and torch.equal(y1, y) and torch.equal(s1, s)
    assert torch.equal(q1.view(torch.uint8), q.view(torch.uint8))
    own = x.clone()
    q2, s2, _, _ = hxq.rmsnorm(own, None, 1e-6, residual=own, sum_out=own)
    q3, s3, _, _ = hxq.rmsnorm(x, None, 1e-6, residual=x)
    assert torch.equal(own, (x.float() * 2).to(x.dtype))
    assert torch.equal(q2.view(torch.uint8), q3.view(torch.uint8)) and torch.equal(s2, s3)


def test_weights_from_the_host_and_other_layouts(hxq):
    """Pageable, pinned, bytes, transposed and sliced weights give what their plain copy gives."""
    import torch
    N, K, M = 260, 700, 33
    xq, xs = make_activation(1, M, K)
    wq, ws = make_weights(2, 3, N, K)
    want = hxq.Fp8Linear(wq[1], ws[1]).forward(xq, xs)
    off = offsets_of([10, 0, 23])
    want_e = hxq.Fp8Linear(wq, ws).forward_grouped(xq, xs, off)
    wide = torch.zeros(N, K + 9, dtype=torch.uint8, device="cuda")
    wide[:, 5:5 + K] = wq[1].view(torch.uint8)
    for W, S in ((wq[1].cpu(), ws[1].cpu()), (wq[1].view(torch.uint8), ws[1].cpu().pin_memory()),
                 (wq[1].view(torch.uint8).cpu().pin_memory(), ws[1]), (wide[:, 5:5 + K], ws[1]),
                 (wq[1].view(torch.uint8).t().contiguous().t(), ws[1].t().contiguous().t())):
        assert torch.equal(hxq.Fp8Linear(W, S).forward(xq, xs), want)
    assert torch.equal(hxq.Fp8Linear(wq.cpu(), ws.cpu()).forward_grouped(xq.view(torch.uint8), xs, off), want_e)


@pytest.mark.parametrize("M", [1, 30, 600])
def test_outputs_and_inputs_at_odd_addresses(hxq, M):
    """y, bias, scales and offsets aligned as their elements only."""
    import torch
    N, K, E = 1024, 640, 3
    xq, xs = make_activation(1, M, K)
    wq, ws = make_weights(2, E, N, K)
    bias = randn(3, E, N)
    counts = [M // 3, 0, M - M // 3]
    off = offsets_of(counts)
    one, ex = hxq.Fp8Linear(wq[0], ws[0]), hxq.Fp8Linear(wq, ws)
    for out, dt in ((hxq.HXQ_OUT_F32, torch.float32), (hxq.HXQ_OUT_BF16, torch.bfloat16)):
        buf = torch.full((M * N + 3,), 7.0, dtype=dt, device="cuda")
        y = buf[1:M * N + 1].view(M, N)
        one.forward(xq, unaligned(xs), bias=unaligned(bias[0]), out_dtype=out, y=y)
        check_product(y, dense_x(xq, xs, K), dense_w(wq[0], ws[0]), bias[0])
        ex.forward_grouped(xq, unaligned(xs), unaligned(off), bias=unaligned(bias), out_dtype=out, y=y)
        at = 0
        for e, n in enumerate(counts):
            if n:
                r = slice(at, at + n)
                check_product(y[r], dense_x(xq[r], xs[r], K), dense_w(wq[e], ws[e]), bias[e])
            at += n
        assert buf[0] == 7 and (buf[M * N + 1:] == 7).all()
    x = randn(5, M, K)
    for f in (lambda q, s: hxq.fp8_quantize(x, q=q, scales=s), lambda q, s: hxq.rmsnorm(x, q=q, scales=s)[:2]):
        a = f(None, None)
        b = f(None, unaligned(a[1]))
        assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("K", [250, 2048, 5000, 33000])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_rmsnorm_residual_without_sum(hxq, dt, K):
    """A NULL sum: the same norm, and neither x nor the residual changes."""
    import torch
    x, res = randn(1, 70, K).to(dtype(dt)), randn(2, 70, K).to(dtype(dt))
    q, s, y, _ = hxq.rmsnorm(x, None, 1e-6, residual=res, want="qy")
    q1, s1, y1 = torch.empty_like(q), torch.empty_like(s), torch.empty_like(y)
    x0, res0, code = x.clone(), res.clone(), hxq.HXQ_TYPE_BF16 if dt == "bf16" else hxq.HXQ_TYPE_F32
    hxq.hxq_rmsnorm(x, code, res, None, code, None, 1e-6, 70, K, y1, q1, s1)
    assert torch.equal(q1.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s1, s) and torch.equal(y1, y)
    assert torch.equal(x, x0) and torch.equal(res, res0)
