"""8-bit-float layers without a GPU: what the entry points refuse, from ctypes
and from plain C, and what the tensor wrappers refuse."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIBDIR = os.path.join(ROOT, "vq_compressed_linear_b200")
BIG = 1 << 31


def _aligned(n, dtype, off=0):
    raw = np.zeros(n * np.dtype(dtype).itemsize + 64 + off, np.uint8)
    start = (-raw.ctypes.data) % 32 + off
    return raw, raw.ctypes.data + start


def test_row_length():
    import vq_compressed_linear_b200 as m
    assert [m.hxq_fp8_ld(k) for k in (1, 15, 16, 17, 128, 11008, 2**31 - 1)] == \
        [16, 16, 16, 32, 128, 11008, 2**31]
    assert m.hxq_fp8_ld(0) == m.HXQ_EINVAL


ROWS = dict(x=True, q=True, s=True, type=0, rows=2, cols=32, xoff=0, qoff=0)
BAD_ROWS = [dict(x=False), dict(q=False), dict(s=False), dict(type=2), dict(type=-1), dict(rows=-1), dict(cols=0),
            dict(cols=-3), dict(rows=BIG), dict(rows=BIG // 2, cols=300), dict(qoff=8), dict(xoff=2), dict(type=1, xoff=1)]


@pytest.mark.parametrize("fn", ["hxq_fp8_quantize", "hxq_fp8_swiglu"])
@pytest.mark.parametrize("bad", BAD_ROWS, ids=str)
def test_quantizers_refuse(fn, bad):
    import vq_compressed_linear_b200 as m
    a = {**ROWS, **bad}
    kx, x = _aligned(512, np.float32, a["xoff"])
    kq, q = _aligned(512, np.uint8, a["qoff"])
    ks, s = _aligned(64, np.float32)
    f = getattr(m.lib, fn)
    assert f(x if a["x"] else None, a["type"], a["rows"], a["cols"], q if a["q"] else None, s if a["s"] else None,
             None) == m.HXQ_EINVAL


@pytest.mark.parametrize("bad", [dict(x=False), dict(q=False), dict(s=False), dict(type=2), dict(E=0), dict(N=0),
                                 dict(K=0), dict(E=1 << 20, N=1 << 20, K=1 << 10)], ids=str)
def test_encode_refuses(bad):
    import vq_compressed_linear_b200 as m
    a = {**dict(x=True, q=True, s=True, type=0, E=1, N=4, K=8), **bad}
    kx, x = _aligned(64, np.float32)
    kq, q = _aligned(64, np.uint8)
    ks, s = _aligned(64, np.float32)
    assert m.lib.hxq_fp8_encode(x if a["x"] else None, a["type"], a["E"], a["N"], a["K"], q if a["q"] else None,
                                s if a["s"] else None, None) == m.HXQ_EINVAL


@pytest.mark.parametrize("bad", [dict(x=False), dict(y=False, q=False, s=False), dict(q=False), dict(s=False),
                                 dict(res=False), dict(xt=3), dict(rt=-1), dict(eps=-1e-6), dict(eps=float("nan")),
                                 dict(eps=float("inf")), dict(rows=-1), dict(cols=0), dict(rows=BIG), dict(qoff=4)],
                         ids=str)
def test_rmsnorm_refuses(bad):
    import vq_compressed_linear_b200 as m
    a = {**dict(x=True, xt=0, res=True, sum=True, rt=0, eps=1e-6, rows=2, cols=32, y=True, q=True, s=True, qoff=0),
         **bad}
    bufs = {k: _aligned(256, np.float32) for k in ("x", "res", "sum", "y", "s")}
    kq, q = _aligned(256, np.uint8, a["qoff"])
    p = {k: (v[1] if a[k] else None) for k, v in bufs.items()}
    assert m.lib.hxq_rmsnorm(p["x"], a["xt"], p["res"], p["sum"], a["rt"], None, a["eps"], a["rows"], a["cols"],
                             p["y"], q if a["q"] else None, p["s"], None) == m.HXQ_EINVAL


@pytest.mark.parametrize("bad", [dict(out=False), dict(w=False), dict(s=False), dict(E=0), dict(E=1025), dict(N=0),
                                 dict(K=0), dict(N=2**31 - 1, K=2**31 - 1), dict(E=1024, N=1 << 17, K=1 << 14)],
                         ids=str)
def test_create_refuses(bad):
    import vq_compressed_linear_b200 as m
    a = {**dict(out=True, w=True, s=True, E=1, N=4, K=8), **bad}
    kw, w = _aligned(64, np.uint8)
    ks, s = _aligned(64, np.float32)
    h = ctypes.c_void_p(7)
    rc = m.lib.hxq_fp8_create(w if a["w"] else None, s if a["s"] else None, a["E"], a["N"], a["K"],
                              ctypes.byref(h) if a["out"] else None)
    assert rc == m.HXQ_EINVAL
    if a["out"]:
        assert h.value is None  # cleared


def test_handle_calls_refuse_null():
    import vq_compressed_linear_b200 as m
    kx, x = _aligned(64, np.float32)
    assert m.lib.hxq_fp8_forward(None, x, x, None, x, 0, 1, None) == m.HXQ_EINVAL
    assert m.lib.hxq_fp8_forward_grouped(None, x, x, x, None, x, 0, 1, None) == m.HXQ_EINVAL
    assert m.lib.hxq_fp8_info(None, None, None, None) == m.HXQ_EINVAL
    assert m.lib.hxq_fp8_check(None) == m.HXQ_EINVAL
    m.lib.hxq_fp8_destroy(None)  # ignored


def test_from_plain_c(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no C compiler")
    exe = tmp_path / "fp8_check"
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "c", "fp8_check.c"), "-o", str(exe),
                    "-L", LIBDIR, "-l:libhxq.so", "-Wl,-rpath," + LIBDIR], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip() == "ok"


def test_wrappers_refuse_host_tensors_and_wrong_types():
    import torch
    import vq_compressed_linear_b200 as m
    for call in (lambda: m.fp8_quantize(torch.zeros(2, 32)), lambda: m.fp8_swiglu(torch.zeros(2, 32)),
                 lambda: m.fp8_encode(torch.zeros(2, 32)), lambda: m.rmsnorm(torch.zeros(2, 32)),
                 lambda: m.Fp8Linear(torch.zeros(2, 32), torch.zeros(1, 1)),
                 lambda: m.Fp8Linear(torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(2, 1))):
        with pytest.raises(m.HXQError) as e:
            call()
        assert e.value.code == m.HXQ_EINVAL
