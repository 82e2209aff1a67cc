"""The gated feed-forward operators without a GPU: their 64-bit references against differences, and the
arguments that the library and its binding refuse before anything is launched."""
import ctypes as C

import numpy as np
import pytest
import torch

import int6_quantized_linear_b200 as ql
from int6_quantized_linear_b200 import _build
from tests import ffn_reference as R

A = 0x10000  # an aligned address that is never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return ql.lib()


@pytest.mark.parametrize("kind", R.ACTS)
def test_activation_gradient_against_differences(kind):
    """Central differences: error h^2 / 6 |f'''| + eps |f| / h, below 1e-8 for h = 1e-5 and |g| <= 8."""
    g = np.linspace(-8, 8, 1601)
    h = 1e-5
    d = (R.act(g + h, kind)[0] - R.act(g - h, kind)[0]) / (2 * h)
    assert np.max(np.abs(d - R.act(g, kind)[1])) < 1e-8


@pytest.mark.parametrize("kind", R.ACTS)
def test_block_gradient_against_differences(kind):
    """dx = dg Wg + du Wu is the gradient of sum(dh * h) in x."""
    rng = np.random.default_rng(5)
    M, F, K = 3, 7, 11
    w, x, dh = rng.normal(size=(2 * F, K)), rng.normal(size=(M, K)), rng.normal(size=(M, F))

    def loss(x):
        gu = x @ w.T
        return np.sum(dh * R.act(gu[:, :F], kind)[0] * gu[:, F:])

    gu = x @ w.T
    dx = R.gated_backward(gu[:, :F], gu[:, F:], dh, kind) @ w
    h = 1e-5
    for m in range(M):
        for k in range(K):
            e = np.zeros_like(x)
            e[m, k] = h
            assert abs((loss(x + e) - loss(x - e)) / (2 * h) - dx[m, k]) < 1e-6


def test_save8_reference():
    """The reference's codes fill seven bits, and a restored value is off by at most half a step."""
    rng = np.random.default_rng(6)
    v = rng.normal(size=(50, 37)) * np.exp(rng.normal(size=(50, 1)) * 20)
    codes, exps = R.save8(v)
    assert codes.shape == (50, 48) and exps.shape == (50, 3)
    top = np.abs(codes.reshape(50, 3, 16).astype(int)).max(-1)
    assert top.min() >= 64 and top.max() <= 127
    step = np.repeat(2.0 ** (exps.astype(int) - 127), 16, axis=1)[:, :37]
    assert np.all(np.abs(R.restore8(codes, exps, 37) - v) <= step / 2)
    assert np.all(codes[:, 37:] == 0)


# ---- refusals ----------------------------------------------------------------------------------------------

def _gated(lib, desc, x=A, M=1, act=0, h=A, saved=(A, A), codes=A, gmeta=A, steps=A, ws=A, ws_bytes=1 << 40):
    d, w = desc.c(), ql.ql_packed(codes, gmeta, steps)
    s = None if saved is None else C.byref(ql.ql_saved8(*saved))
    return lib.qlinear_gated(C.byref(d), C.byref(w), x, M, act, h, s, ws, ws_bytes, None)


def test_gated_refusals(lib):
    d = ql.Desc("int4", 64, 256)
    assert _gated(lib, ql.Desc("int4", 63, 256)) == ql.QL_ERR_SHAPE          # an odd number of rows
    assert _gated(lib, ql.Desc("int4", 64, 200)) == ql.QL_ERR_SHAPE          # K of the format
    assert _gated(lib, ql.Desc("affine", 64, 96, 4, 32)) == ql.QL_ERR_SHAPE  # K % 64
    for bad in (-1, 3, 99):
        assert _gated(lib, d, act=bad) == ql.QL_ERR_UNSUPPORTED
    for bad in (0, -1, 1 << 31):
        assert _gated(lib, d, M=bad) == ql.QL_ERR_RANGE
    for k in ("x", "h", "codes", "gmeta", "steps", "ws"):
        assert _gated(lib, d, **{k: None}) == ql.QL_ERR_NULL, k
        assert _gated(lib, d, **{k: A + 8}) == ql.QL_ERR_ALIGN, k
    assert _gated(lib, d, ws=A + 16) == ql.QL_ERR_ALIGN                      # the workspace wants 256
    for s, want in (((None, A), ql.QL_ERR_NULL), ((A, None), ql.QL_ERR_NULL), ((A + 8, A), ql.QL_ERR_ALIGN),
                    ((A, A + 8), ql.QL_ERR_ALIGN)):
        assert _gated(lib, d, saved=s) == want
    need = ql.qlinear_gated_workspace_bytes(d, 1)
    assert _gated(lib, d, ws_bytes=need - 1) == ql.QL_ERR_SHAPE
    bad = ql.ql_desc(9, 0, 0, 0, 64, 256)
    n = C.c_size_t()
    assert lib.qlinear_gated_workspace_bytes(C.byref(bad), 1, C.byref(n)) == ql.QL_ERR_UNSUPPORTED
    assert lib.qlinear_gated_workspace_bytes(None, 1, C.byref(n)) == ql.QL_ERR_NULL


def _dx(lib, desc, dy=A, M=1, dx=A, codes=A, gmeta=A, steps=A, ws=A, ws_bytes=1 << 40):
    d, w = desc.c(), ql.ql_packed(codes, gmeta, steps)
    return lib.qlinear_gemm_dx(C.byref(d), C.byref(w), dy, M, dx, ws, ws_bytes, None)


def _backward(lib, desc, dh=A, M=1, act=0, dgu=A, dx=A, saved=(A, A), codes=A, gmeta=A, steps=A, ws=A,
              ws_bytes=1 << 40):
    d, w = desc.c(), ql.ql_packed(codes, gmeta, steps)
    s = None if saved is None else C.byref(ql.ql_saved8(*saved))
    return lib.qlinear_gated_backward(C.byref(d), C.byref(w), s, dh, M, act, dgu, dx, ws, ws_bytes, None)


@pytest.mark.parametrize("call,ptrs", [(_dx, ("dy", "dx", "codes", "gmeta", "steps", "ws")),
                                       (_backward, ("dh", "dx", "codes", "gmeta", "steps", "ws"))])
def test_dx_refusals(lib, call, ptrs):
    d = ql.Desc("int6", 64, 512)
    assert call(lib, ql.Desc("int6", 64, 384)) == ql.QL_ERR_SHAPE
    assert call(lib, ql.Desc("int6", (1 << 31) - 8, 256)) == ql.QL_ERR_SHAPE
    for bad in (0, -5, 1 << 31):
        assert call(lib, d, M=bad) == ql.QL_ERR_RANGE
    for k in ptrs:
        assert call(lib, d, **{k: None}) == ql.QL_ERR_NULL, k
        assert call(lib, d, **{k: A + 8}) == ql.QL_ERR_ALIGN, k
    need = ql.qlinear_gemm_dx_workspace_bytes(d, 1)
    assert call(lib, d, ws_bytes=need - 1) == ql.QL_ERR_SHAPE


def test_backward_refusals(lib):
    d = ql.Desc("affine", 64, 512, 4, 64)
    assert _backward(lib, ql.Desc("affine", 65, 512, 4, 64)) == ql.QL_ERR_SHAPE
    assert _backward(lib, d, act=7) == ql.QL_ERR_UNSUPPORTED
    assert _backward(lib, d, saved=None) == ql.QL_ERR_NULL
    assert _backward(lib, d, saved=(A, None)) == ql.QL_ERR_NULL
    assert _backward(lib, d, saved=(A + 4, A)) == ql.QL_ERR_ALIGN
    assert _backward(lib, d, dgu=A + 2) == ql.QL_ERR_ALIGN


def test_saved8_refusals(lib):
    s = ql.ql_saved8(A, A)
    c, e = C.c_size_t(), C.c_size_t()
    for rows, cols in ((0, 5), (5, 0), (-1, 5)):
        assert lib.qlinear_saved8_bytes(rows, cols, C.byref(c), C.byref(e)) == ql.QL_ERR_SHAPE
        assert lib.qlinear_save8(A, rows, cols, C.byref(s), None) == ql.QL_ERR_SHAPE
    for rows, cols in ((1 << 38, 17), (1, (1 << 38) + 1), (1 << 62, 1 << 62), (1, (1 << 63) - 1)):
        assert lib.qlinear_saved8_bytes(rows, cols, C.byref(c), C.byref(e)) == ql.QL_ERR_RANGE
        assert lib.qlinear_restore8(C.byref(s), rows, cols, A, None) == ql.QL_ERR_RANGE
    assert lib.qlinear_saved8_bytes(3, 5, None, C.byref(e)) == ql.QL_ERR_NULL
    assert lib.qlinear_save8(None, 3, 5, C.byref(s), None) == ql.QL_ERR_NULL
    assert lib.qlinear_save8(A, 3, 5, None, None) == ql.QL_ERR_NULL
    assert lib.qlinear_save8(A + 2, 3, 5, C.byref(s), None) == ql.QL_ERR_ALIGN
    assert lib.qlinear_restore8(C.byref(ql.ql_saved8(A, A + 4)), 3, 5, A, None) == ql.QL_ERR_ALIGN
    assert lib.qlinear_restore8(C.byref(ql.ql_saved8(None, A)), 3, 5, A, None) == ql.QL_ERR_NULL
    assert ql.qlinear_saved8_bytes(3, 5) == (3 * 16, 3)
    assert ql.qlinear_saved8_bytes(2, 32) == (2 * 32, 4)


def _a256(n):
    return (n + 255) // 256 * 256


@pytest.mark.parametrize("fmt,bits,group,N,K,M", [("int4", 0, 0, 27648, 5120, 2048), ("int6", 0, 0, 100, 256, 1),
                                                  ("affine", 8, 128, 77, 640, 33), ("int6p", 0, 0, 65, 512, 32)])
def test_dx_workspace_formula(lib, fmt, bits, group, N, K, M):
    np_ = (N + 63) // 64 * 64
    run = group if fmt == "affine" else 32
    tiles = -(-M // (32 if M <= 32 else 64 if M <= 64 else 256))
    tokens = -(-(-(-M // tiles)) // 16) * 16  # M spread evenly, rounded up to 16
    want = (_a256(2 * M * np_) + _a256(4 * M) + _a256(np_) + _a256(4 * (K // run) * np_)
            + 148 * 1024 * tokens * (2 if M <= 64 else 1))
    assert ql.qlinear_gemm_dx_workspace_bytes(ql.Desc(fmt, N, K, bits, group), M) == want


def test_gated_workspace_covers_both_forms(lib):
    for d, M in ((ql.Desc("int4", 64, 256), 1), (ql.Desc("affine", 14336, 4096, 2, 64), 32)):
        n = ql.qlinear_gated_workspace_bytes(d, M)
        assert n == max(ql.qlinear_gemm_workspace_bytes(d, M), ql.qlinear_gemv_workspace_bytes(d, M))
    d = ql.Desc("int4", 64, 256)
    assert ql.qlinear_gated_workspace_bytes(d, 9) == ql.qlinear_gemm_workspace_bytes(d, 9)


def test_binding_refuses_host_tensors(lib):
    """The binding checks its tensors before the library sees a pointer."""
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    d = ql.Desc("int4", 32, 256)
    w = [torch.zeros(n, dtype=torch.uint8) for n in ql.qlinear_packed_bytes(d)]
    saved = ql.alloc_saved8(2, 16, "cpu")
    for call in (lambda: ql.qlinear_gated(d, *w, bf(1, 256), 1, "silu", bf(1, 16)),
                 lambda: ql.qlinear_gemm_dx(d, *w, bf(1, 32), 1, bf(1, 256)),
                 lambda: ql.qlinear_gated_backward(d, *w, saved, bf(1, 16), 1, "silu", bf(1, 256)),
                 lambda: ql.qlinear_save8(bf(2, 16), 2, 16, saved),
                 lambda: ql.qlinear_restore8(saved, 2, 16, bf(2, 16))):
        with pytest.raises(ql.QLinearError) as e:
            call()
        assert e.value.status == ql.QL_ERR_UNSUPPORTED
    with pytest.raises(ql.QLinearError) as e:
        ql.qlinear_gated(d, *w, bf(1, 256), 1, "tanh", bf(1, 16))
    assert e.value.status == ql.QL_ERR_UNSUPPORTED


@pytest.mark.parametrize("call", [_dx, _backward])
def test_dx_refuses_what_its_grids_cannot_count(lib, call):
    """K above 2^26 (the metadata pass's grid) or M * K above 2^40 (tiles counted in 32 bits); the largest that
    fit are accepted (their workspace is worked out)."""
    most = 1 << 26
    n = C.c_size_t()
    for K, M in ((most + 256, 1), (1 << 30, 1), (most, (1 << 14) + 1), (1 << 20, (1 << 20) + 1)):
        d = ql.Desc("int4", 64, K)
        assert call(lib, d, M=M) == ql.QL_ERR_RANGE
        assert lib.qlinear_gemm_dx_workspace_bytes(C.byref(d.c()), M, C.byref(n)) == ql.QL_ERR_RANGE
    for K, M in ((most, 1 << 14), (1 << 20, 1 << 20)):
        assert ql.qlinear_gemm_dx_workspace_bytes(ql.Desc("int4", 64, K), M) > 2 * M * 64


def test_gated_refuses_rows_past_32_bits(lib):
    """k is a 32-bit coordinate of the copies."""
    d = ql.Desc("int4", 64, 1 << 31)
    assert _gated(lib, d) == ql.QL_ERR_SHAPE
    n = C.c_size_t()
    assert lib.qlinear_gated_workspace_bytes(C.byref(d.c()), 1, C.byref(n)) == ql.QL_ERR_SHAPE
