"""Host-side tests of the 4-bit operators and the table lookup: refusals (which come before any device work), the
reference definitions themselves, and the workspace size.  No GPU needed."""
from __future__ import annotations

import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import int8_gemm_b200 as bs
import lowbit_ref as ref
from int8_gemm_b200 import build as bsbuild

HAS_GPU = torch.cuda.is_available()
P = 1 << 20  # a fake, aligned "device" address: never dereferenced
v = ctypes.c_void_p


@pytest.fixture(scope="module", autouse=True)
def built_library():
    bsbuild.build()
    return bs.lib()


def _quant(**kw):
    a = dict(x=P, xd=0, N=10, K=301, ldx=304, q=P, ldq=160, s=P, sd=1, lds=5, z=None, ldz=0, group=64)
    a.update(kw)
    return bs.lib().bs_quantize_int4(v(a["x"]), a["xd"], a["N"], a["K"], a["ldx"], v(a["q"]), a["ldq"], v(a["s"]), a["sd"],
                                     a["lds"], v(a["z"]), a["ldz"], a["group"], None)


def _deq(**kw):
    a = dict(q=P, ldq=160, s=P, sd=1, lds=5, z=None, ldz=0, group=64, out=P, od=0, ldo=304, N=10, K=301)
    a.update(kw)
    return bs.lib().bs_dequantize_int4(v(a["q"]), a["ldq"], v(a["s"]), a["sd"], a["lds"], v(a["z"]), a["ldz"], a["group"],
                                       v(a["out"]), a["od"], a["ldo"], a["N"], a["K"], None)


def _gemv(**kw):
    a = dict(x=P, xd=0, ldx=304, q=P, ldq=160, s=P, sd=1, lds=5, z=None, ldz=0, group=64, bias=None, out=P, od=0, ldo=10,
             M=4, N=10, K=301)
    a.update(kw)
    return bs.lib().bs_gemv_int4(v(a["x"]), a["xd"], a["ldx"], v(a["q"]), a["ldq"], v(a["s"]), a["sd"], a["lds"], v(a["z"]),
                                 a["ldz"], a["group"], v(a["bias"]), v(a["out"]), a["od"], a["ldo"], a["M"], a["N"], a["K"],
                                 None)


@pytest.mark.parametrize("call", [_quant, _deq, _gemv])
def test_int4_matrix_refusals(call):
    assert call(N=-1) == bs.BS_ERR_SHAPE and call(K=-1) == bs.BS_ERR_SHAPE
    assert call(N=1 << 31) == bs.BS_ERR_SHAPE and call(K=1 << 31) == bs.BS_ERR_SHAPE
    for g in (0, -32, 16, 96, 256):
        assert call(group=g) == bs.BS_ERR_SHAPE
    assert call(sd=2) == bs.BS_ERR_DTYPE
    assert call(q=0) == bs.BS_ERR_NULL and call(s=0) == bs.BS_ERR_NULL
    assert call(ldq=150) == bs.BS_ERR_LAYOUT  # ceil(301 / 2) = 151
    assert call(lds=4) == bs.BS_ERR_LAYOUT    # ceil(301 / 64) = 5
    assert call(z=P, ldz=4) == bs.BS_ERR_LAYOUT
    assert call(ldq=1 << 61) == bs.BS_ERR_LAYOUT and call(lds=1 << 60) == bs.BS_ERR_LAYOUT
    assert call(s=P + 2) == bs.BS_ERR_ALIGNMENT and call(sd=0, s=P + 1) == bs.BS_ERR_ALIGNMENT
    assert call(N=0) == bs.BS_OK
    if not HAS_GPU:  # well-formed calls reach the device check (never launched with fake pointers on a GPU)
        assert call() == bs.BS_ERR_DEVICE and call(z=P + 1, ldz=5, sd=0, s=P + 2) == bs.BS_ERR_DEVICE


def test_quantize_refusals():
    assert _quant(K=0) == bs.BS_OK
    assert _quant(xd=2) == bs.BS_ERR_DTYPE and _quant(x=0) == bs.BS_ERR_NULL
    assert _quant(ldx=300) == bs.BS_ERR_LAYOUT
    assert _quant(x=P + 1) == bs.BS_ERR_ALIGNMENT and _quant(xd=1, x=P + 2) == bs.BS_ERR_ALIGNMENT
    if not HAS_GPU:
        assert _quant(q=P + 1, ldq=151, x=P + 2, ldx=301) == bs.BS_ERR_DEVICE  # any alignment of codes and rows


def test_dequantize_refusals():
    assert _deq(K=0) == bs.BS_OK
    assert _deq(od=2) == bs.BS_ERR_DTYPE and _deq(od=3) == bs.BS_ERR_DTYPE
    assert _deq(out=0) == bs.BS_ERR_NULL and _deq(ldo=300) == bs.BS_ERR_LAYOUT
    assert _deq(out=P + 1) == bs.BS_ERR_ALIGNMENT and _deq(od=1, out=P + 2) == bs.BS_ERR_ALIGNMENT


def test_gemv_refusals():
    assert _gemv(M=-1) == bs.BS_ERR_SHAPE and _gemv(M=33) == bs.BS_ERR_SHAPE
    assert "32" in bs.lib().bs_last_error_message().decode()
    assert _gemv(M=0) == bs.BS_OK
    assert _gemv(xd=2) == bs.BS_ERR_DTYPE and _gemv(od=2) == bs.BS_ERR_DTYPE
    assert _gemv(x=0) == bs.BS_ERR_NULL and _gemv(out=0) == bs.BS_ERR_NULL
    assert _gemv(ldx=300) == bs.BS_ERR_LAYOUT and _gemv(ldo=9) == bs.BS_ERR_LAYOUT
    assert _gemv(q=P + 8) == bs.BS_ERR_ALIGNMENT and _gemv(ldq=152) == bs.BS_ERR_ALIGNMENT
    assert _gemv(x=P + 1) == bs.BS_ERR_ALIGNMENT and _gemv(bias=P + 2) == bs.BS_ERR_ALIGNMENT
    assert _gemv(out=P + 1) == bs.BS_ERR_ALIGNMENT
    if not HAS_GPU:
        assert _gemv(x=P + 2, ldx=301, out=P + 2, ldo=11) == bs.BS_ERR_DEVICE
        assert _gemv(K=0, x=0, q=0, s=0, ldo=10) == bs.BS_ERR_DEVICE  # nothing of K = 0 is read


def _emb(**kw):
    a = dict(tok=P, td=1, T=7, table=P, fmt=0, ld=300, s=None, sd=1, lds=0, z=None, ldz=0, group=64, V=50, D=300, alpha=1.0,
             out=P, od=0, ldo=300)
    a.update(kw)
    return bs.lib().bs_embedding(v(a["tok"]), a["td"], a["T"], v(a["table"]), a["fmt"], a["ld"], v(a["s"]), a["sd"], a["lds"],
                                 v(a["z"]), a["ldz"], a["group"], a["V"], a["D"], a["alpha"], v(a["out"]), a["od"], a["ldo"],
                                 None)


def test_embedding_refusals():
    for k in ("T", "V", "D"):
        assert _emb(**{k: -1}) == bs.BS_ERR_SHAPE and _emb(**{k: 1 << 31}) == bs.BS_ERR_SHAPE
    assert _emb(td=2) == bs.BS_ERR_DTYPE and _emb(fmt=5) == bs.BS_ERR_DTYPE and _emb(fmt=-1) == bs.BS_ERR_DTYPE
    assert _emb(od=2) == bs.BS_ERR_DTYPE
    assert _emb(tok=0) == bs.BS_ERR_NULL and _emb(table=0) == bs.BS_ERR_NULL and _emb(out=0) == bs.BS_ERR_NULL
    assert _emb(ld=299) == bs.BS_ERR_LAYOUT and _emb(ldo=299) == bs.BS_ERR_LAYOUT and _emb(ld=1 << 60) == bs.BS_ERR_LAYOUT
    assert _emb(tok=P + 4) == bs.BS_ERR_ALIGNMENT and _emb(table=P + 1) == bs.BS_ERR_ALIGNMENT
    assert _emb(fmt=1, table=P + 2) == bs.BS_ERR_ALIGNMENT and _emb(out=P + 1) == bs.BS_ERR_ALIGNMENT
    assert _emb(fmt=2) == bs.BS_ERR_NULL and _emb(fmt=2, s=P, lds=2) == bs.BS_ERR_LAYOUT  # ceil(300 / 128) = 3
    assert _emb(fmt=2, s=P + 2, lds=3) == bs.BS_ERR_ALIGNMENT
    assert _emb(fmt=4, ld=150) == bs.BS_ERR_NULL and _emb(fmt=4, ld=149, s=P, lds=5) == bs.BS_ERR_LAYOUT
    assert _emb(fmt=4, ld=150, s=P, lds=4) == bs.BS_ERR_LAYOUT and _emb(fmt=4, ld=150, s=P, lds=5, group=48) == bs.BS_ERR_SHAPE
    assert _emb(T=0) == bs.BS_OK and _emb(D=0) == bs.BS_OK
    if not HAS_GPU:
        for kw in ({}, {"td": 0, "tok": P + 4}, {"V": 0, "table": 0}, {"fmt": 3, "s": P + 1, "lds": 3},
                   {"fmt": 4, "ld": 150, "s": P, "lds": 5, "table": P + 1}):
            assert _emb(**kw) == bs.BS_ERR_DEVICE, kw


def test_outputs_below_2_to_the_43_elements():
    """Rows times columns, the columns counted up to a multiple of 4."""
    for call in (lambda rows, cols: _emb(T=rows, D=cols, ld=cols, ldo=cols),
                 lambda rows, cols: _deq(N=rows, K=cols, ldq=cols, lds=cols, ldo=cols),
                 lambda rows, cols: _grad(V=rows, D=cols, ldg=cols, ldd=cols, n=1 << 62)):
        assert call(1 << 29, 1 << 14) == bs.BS_ERR_SHAPE
        assert "2^43" in bs.lib().bs_last_error_message().decode()
        assert call(1 << 30, (1 << 13) - 3) == bs.BS_ERR_SHAPE
        if not HAS_GPU:
            assert call((1 << 29) - 1, 1 << 14) == bs.BS_ERR_DEVICE


def _grad(**kw):
    a = dict(tok=P, td=1, T=2000, grad=P, gd=0, ldg=300, V=50, D=300, alpha=1.0, pad=-1, d=P, od=1, ldd=300, acc=0, ws=P,
             n=None)
    a.update(kw)
    n = bs.lib().bs_embedding_grad_workspace(2000, 50, 300) if a["n"] is None else a["n"]
    return bs.lib().bs_embedding_grad(v(a["tok"]), a["td"], a["T"], v(a["grad"]), a["gd"], a["ldg"], a["V"], a["D"],
                                      a["alpha"], a["pad"], v(a["d"]), a["od"], a["ldd"], a["acc"], v(a["ws"]), n, None)


def test_embedding_grad_refusals():
    for k in ("T", "V", "D"):
        assert _grad(**{k: -1}) == bs.BS_ERR_SHAPE and _grad(**{k: 1 << 31}) == bs.BS_ERR_SHAPE
    assert _grad(td=2) == bs.BS_ERR_DTYPE and _grad(gd=2) == bs.BS_ERR_DTYPE and _grad(od=2) == bs.BS_ERR_DTYPE
    for k in ("tok", "grad", "d", "ws"):
        assert _grad(**{k: 0}) == bs.BS_ERR_NULL, k
    assert _grad(ldg=299) == bs.BS_ERR_LAYOUT and _grad(ldd=299) == bs.BS_ERR_LAYOUT
    assert _grad(tok=P + 4) == bs.BS_ERR_ALIGNMENT and _grad(grad=P + 1) == bs.BS_ERR_ALIGNMENT
    assert _grad(d=P + 2) == bs.BS_ERR_ALIGNMENT and _grad(ws=P + 16) == bs.BS_ERR_ALIGNMENT
    assert _grad(n=1024) == bs.BS_ERR_WORKSPACE
    assert _grad(V=0) == bs.BS_OK and _grad(D=0) == bs.BS_OK
    if not HAS_GPU:
        assert _grad() == bs.BS_ERR_DEVICE and _grad(T=0, tok=0, grad=0, ws=0, n=0) == bs.BS_ERR_DEVICE
        assert _grad(T=512, ws=0, n=0) == bs.BS_ERR_DEVICE


def test_embedding_grad_workspace_covers_pairs_and_partials():
    size = bs.lib().bs_embedding_grad_workspace
    assert size(0, 100, 64) == 0 and size(-1, 5, 5) == 0 and size(5, 1 << 31, 5) == 0
    assert size(1, 100, 64) == 0 and size(512, 100, 64) == 0  # few tokens need none
    for T, D in ((513, 1), (1100, 7), (16640, 5120)):
        assert size(T, 1000, D) >= 16 * T + 2 * -(-T // 32) * 4 * D
        assert size(T, 1000, D) == size(T, 5, D)
    assert size(2**31 - 1, 2**31 - 1, 2**31 - 1) > 2**58


def test_lookup_kernels_keep_their_pieces_in_registers(tmp_path):
    """No lookup kernel spills, but for those of 4-bit tables, where fewer pieces per lane measured slower."""
    src = os.path.join(bsbuild.CSRC, "kernels_lookup.cu")
    cmd = [bsbuild.nvcc(), *bsbuild.NVCC_FLAGS, "-Xptxas", "-v", "-c", src, "-o", str(tmp_path / "lookup.o")]
    log = subprocess.run(cmd, capture_output=True, text=True, check=True).stderr
    found = re.findall(r"Function properties for \S*lookup_kernelILNS0_3FmtE(\d)E(\S+)\n.*?(\d+) bytes spill stores", log)
    assert len(found) == 5 * 2 * 2, log  # formats, output types, small and large
    for fmt, rest, spilled in found:
        assert int(spilled) <= (64 if fmt == "4" else 0), (fmt, rest, spilled)


def test_binding_rejects_cpu_tensors():
    x = torch.zeros(4, 64)
    q, s = torch.zeros(8, 32, dtype=torch.uint8), torch.ones(8, 1)
    t = torch.zeros(3, dtype=torch.int64)
    for call in (lambda: bs.bs_quantize_int4(x), lambda: bs.bs_dequantize_int4(q, s), lambda: bs.bs_gemv_int4(x, q, s),
                 lambda: bs.bs_embedding(t, x), lambda: bs.bs_embedding_grad(t, x[:3], 5)):
        with pytest.raises(bs.BsgemmError) as e:
            call()
        assert e.value.status == bs.BS_ERR_DEVICE


# ---------------------------------------------------------------------------
# the definitions that the GPU tests compare with
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("asym", [False, True])
@pytest.mark.parametrize("group,K", [(32, 64), (64, 130), (128, 127)])
def test_reference_quantiser_properties(group, K, asym):
    g = torch.Generator().manual_seed(5)
    x = torch.randn(9, K, generator=g) * torch.tensor([1e-3, 1, 50.0])[torch.arange(9) % 3][:, None]
    x[4] = 0
    x[5, 3:] = 0
    codes, scale, zero = ref.quantize_int4(x, group, False, asym)
    assert codes.min() >= 0 and codes.max() <= 15 and zero.min() >= 0 and zero.max() <= 15
    q = ref.pack(codes, zero, group)
    assert np.array_equal(ref.unpack(q, K), codes)
    val = ref.values(codes, scale, zero, group)
    # half a step (and one more unit for the rounding of the zero point) from the input, zero exactly kept
    step = ref.spread(scale, group, K)
    assert np.all(np.abs(val - x.numpy()) <= step * (1.0 if asym else 0.5) * (1 + 2**-20))
    assert np.all(val[x.numpy() == 0] == 0) and np.all(scale[4] == 1)
    if not asym:
        assert codes.min() >= 1


def test_reference_gradient_is_the_lookup_s():
    rng = np.random.default_rng(3)
    table = rng.integers(-8, 8, (6, 5)).astype(np.float32)
    tokens = np.array([0, 3, 3, 5, 9, -1, 0, 0])
    c = rng.integers(-8, 8, (8, 5)).astype(np.float32)
    d, S, n = ref.lookup_grad(tokens, c, 6, 2.0)
    for r in range(6):
        for j in range(5):
            up = table.copy()
            up[r, j] += 1
            # the loss sum(c * lookup) is linear in the table, so a difference is its derivative
            assert np.sum(c * ref.lookup(tokens, up, 2.0)) - np.sum(c * ref.lookup(tokens, table, 2.0)) == d[r, j]
    assert n.tolist() == [3, 0, 0, 2, 0, 1] and np.all(S >= np.abs(d))


@pytest.mark.parametrize("div,r", [(7, float.fromhex("0x1.24924ap-3")), (15, float.fromhex("0x1.111112p-4"))])
def test_quotients_by_the_range_constants(div, r):
    """The quantiser's a / 7 and a / 15 (a constant reciprocal and Markstein's correction step) for every significand;
    the steps scale with the exponent where nothing under- or overflows.  The fma is taken in extended precision."""
    assert np.float32(r) == np.float32(1) / np.float32(div) and np.finfo(np.longdouble).nmant >= 63
    for lo in range(0, 1 << 23, 1 << 20):
        a = (np.arange(lo, lo + (1 << 20), dtype=np.int64) + (1 << 23)).astype(np.float32) * np.float32(2.0**-23)
        q1 = (a * np.float32(r)).astype(np.float32)
        rem = a.astype(np.float64) - q1.astype(np.float64) * div  # exact, and an fp32 number
        assert np.array_equal(rem, rem.astype(np.float32))
        q = (q1.astype(np.longdouble) + rem.astype(np.longdouble) * np.longdouble(r)).astype(np.float32)
        assert np.array_equal(q, a / np.float32(div))
