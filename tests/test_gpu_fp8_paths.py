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
