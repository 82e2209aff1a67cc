"""The gated feed-forward block, its backward pass, 8-bit checkpoints and input gradients against 64-bit
references built on the CPU oracle's weights (GPU only).

Tolerances.  A product's accumulator is held to the library's stated budget (tests/gpu_helpers): 1e-2 rms of
the exact result plus 1e-3 -- the operands' fp16 rounding moves it by about 1e-3 rms, so this is ten of its
standard deviations.  The activations here are scaled so that rms(g) is about 2, so the absolute 1e-3 is left
out.  From eps_g, eps_u of the two accumulators,
    |h - h_ref| <= |u| max|act'| eps_g + |act(g)| eps_u + max|act'| eps_g eps_u + half a bf16 step of h,
with |act'| <= 1.13 for the three activations, and the rms of g and u that of their distribution, 2, where few
of them are drawn.  Over an output of a thousand values and more the errors average out: the norm of the error
is held to 4e-3 of the result's, a bf16 rounding being 1.7e-3 (uniform in half a step of 2^-9 .. 2^-8 relative)
and the operands' 1e-3 entering up to three times.
"""
import numpy as np
import pytest
import torch

import int6_quantized_linear_b200 as ql
from tests import ffn_reference as R
from tests.gpu_helpers import Layer, bf16_to_f64, dev, half_ulp_bf16, host

pytestmark = pytest.mark.gpu

FORMATS = [("int4", 0, 0), ("int6", 0, 0), ("int6p", 0, 0), ("affine", 2, 64), ("affine", 4, 32), ("affine", 4, 64),
           ("affine", 8, 32), ("affine", 8, 128)]
MAX_SLOPE = 1.13


def bf16(a: np.ndarray) -> np.ndarray:
    """float64 -> bf16 bits, nearest-even."""
    return torch.from_numpy(a).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def to_dev(bits):
    return dev(bits).view(torch.bfloat16)


def out(rows, cols):
    """A bf16 output with a row of canaries before and after it."""
    full = torch.full(((rows + 2) * cols + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    start = -(-cols // 8) * 8
    return full, full[start:start + rows * cols].view(rows, cols)


def untouched(full, rows, cols):
    start = -(-cols // 8) * 8
    return bool((full[:start] == 7).all()) and bool((full[start + rows * cols:] == 7).all())


def f64(t: torch.Tensor) -> np.ndarray:
    return bf16_to_f64(host(t.contiguous().view(torch.int16), np.uint16))


def layer(fmt, N, K, seed, bits=0, group=0):
    L = Layer(fmt, N, K, seed, bits, group)
    L.wref = L.oracle_w().astype(np.float64)
    return L


def scaled_x(L, M, seed, rms=2.0):
    """bf16 x for which the products have about the given rms."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(M, L.K)) * rms / np.sqrt(np.mean(L.wref ** 2) * L.K)
    return bf16(x)


def rms(a):
    return float(np.sqrt(np.mean(a ** 2)))


def close(got, ref, tol, what):
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    bad = np.abs(got - ref) > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, worst {np.max(np.abs(got - ref) / tol):.2f} tolerances"
    n = np.linalg.norm(ref)
    assert ref.size < 1000 or np.linalg.norm(got - ref) <= 4e-3 * n + 1e-30, f"{what}: norm of the error {np.linalg.norm(got - ref) / n:.2e}"


def check_h(h, g, u, kind, what):
    a, _ = R.act(g, kind)
    eg, eu = 1e-2 * max(2.0, rms(g)), 1e-2 * max(2.0, rms(u))
    close(h, a * u, np.abs(u) * MAX_SLOPE * eg + np.abs(a) * eu + MAX_SLOPE * eg * eu + half_ulp_bf16(a * u), what)


def check_dx(dx, d, w, what):
    ref = d @ w
    close(dx, ref, 1e-2 * rms(ref) + half_ulp_bf16(ref), what)


def run_gated(L, xb, M, kind, save=False):
    F = L.N // 2
    full, h = out(M, F)
    saved = ql.alloc_saved8(2 * M, F) if save else None
    ql.qlinear_gated(L.desc, *L.packed(), to_dev(xb), M, kind, h, saved=saved)
    assert ql.qlinear_sync_status() == ql.QL_OK
    assert untouched(full, M, F)
    return h, saved


# ---- forward -----------------------------------------------------------------------------------------------

@pytest.mark.parametrize("M", [1, 2, 3, 8, 9, 17, 32, 33, 77, 300])
@pytest.mark.parametrize("fmt,bits,group", FORMATS)
def test_gated(cuda, fmt, bits, group, M):
    """Every form by its token count, features that end inside a tile, K of a few blocks."""
    F, K, kind = 150, 512, R.ACTS[M % 3]
    L = layer(fmt, 2 * F, K, 100 + M, bits, group)
    xb = scaled_x(L, M, M)
    h, _ = run_gated(L, xb, M, kind)
    gu = bf16_to_f64(xb) @ L.wref.T
    check_h(f64(h), gu[:, :F], gu[:, F:], kind, f"{fmt}{bits} M={M}")


@pytest.mark.parametrize("F", [1, 15, 16, 31, 32, 33, 64, 65, 1003])
@pytest.mark.parametrize("M", [1, 4, 20, 40])
def test_gated_feature_counts(cuda, F, M):
    L = layer("int4", 2 * F, 768, F, 0, 0)
    xb = scaled_x(L, M, F + M)
    h, _ = run_gated(L, xb, M, "silu")
    gu = bf16_to_f64(xb) @ L.wref.T
    check_h(f64(h), gu[:, :F], gu[:, F:], "silu", f"F={F} M={M}")


# F and K at which the decode kernels cut K in parts, leave it whole, or cut some row groups only (444 or 296
# resident CTAs of 32 features), and the GEMM has more tiles than SMs
@pytest.mark.parametrize("fmt,bits,group,M,F,K", [
    ("int4", 0, 0, 1, 64, 8192), ("int4", 0, 0, 1, 14300, 256), ("int4", 0, 0, 1, 13824, 768),
    ("int4", 0, 0, 5, 64, 8192), ("int4", 0, 0, 5, 14300, 256), ("int4", 0, 0, 5, 13824, 768),
    ("int4", 0, 0, 8, 14300, 512), ("int4", 0, 0, 25, 9700, 256), ("int4", 0, 0, 300, 9700, 256),
    ("int6", 0, 0, 1, 14300, 256), ("int6", 0, 0, 8, 13824, 512), ("int6p", 0, 0, 4, 13824, 512),
    ("affine", 4, 64, 1, 14300, 256), ("affine", 4, 64, 3, 9700, 256), ("affine", 8, 64, 24, 9700, 256),
    ("affine", 2, 32, 12, 9700, 512), ("affine", 8, 128, 1, 9700, 256)])
def test_gated_splits(cuda, fmt, bits, group, M, F, K):
    L = layer(fmt, 2 * F, K, 7, bits, group)
    xb = scaled_x(L, M, 8)
    h, _ = run_gated(L, xb, M, "gelu_tanh")
    gu = bf16_to_f64(xb) @ L.wref.T
    check_h(f64(h), gu[:, :F], gu[:, F:], "gelu_tanh", f"{fmt} M={M} F={F} K={K}")


def test_gated_outlier_tokens(cuda):
    """A dominant element in x: the decode kernels' 24-bit fixed point."""
    L = layer("int4", 300, 1024, 3)
    for M in (1, 4):
        x = bf16_to_f64(scaled_x(L, M, 4))
        x[:, 17] *= 3000.0
        xb = bf16(x)
        gu = bf16_to_f64(xb) @ L.wref.T
        h, _ = run_gated(L, xb, M, "gelu")
        check_h(f64(h), gu[:, :150], gu[:, 150:], "gelu", f"outlier M={M}")


def test_gated_is_what_stacking_makes(cuda):
    """Two packed layers stacked by qlinear_concat_n are the block's layer."""
    F, K, M = 200, 1024, 70
    A, B = layer("int6", F, K, 11), layer("int6", F, K, 12)
    d = ql.Desc("int6", 2 * F, K)
    w = ql.alloc_packed(d)
    ql.qlinear_concat_n(A.desc, A.packed(), B.desc, B.packed(), w)
    xb = scaled_x(A, M, 13)
    h = torch.empty((M, F), dtype=torch.bfloat16, device="cuda")
    ql.qlinear_gated(d, *w, to_dev(xb), M, "silu", h)
    assert ql.qlinear_sync_status() == ql.QL_OK
    x = bf16_to_f64(xb)
    check_h(f64(h), x @ A.wref.T, x @ B.wref.T, "silu", "stacked")


# ---- 8-bit form --------------------------------------------------------------------------------------------

def special_rows(cols, seed):
    """bf16 rows with zeros, subnormals, extremes, borders of the scale and values that are not finite."""
    rng = np.random.default_rng(seed)
    v = rng.normal(size=(24, cols)) * np.exp2(rng.integers(-130, 127, size=(24, 1)).astype(np.float64))
    b = bf16(v)
    b[1] = 0
    b[2] = 0x8000
    b[3] = rng.integers(0, 0x80, cols)                 # subnormals
    b[4] = 0x42FE + rng.integers(0, 3, cols)           # 127, 127.5, 128
    b[5] = 0x7F7F                                      # the largest finite bf16
    b[6] = 0x7F7E
    b[7, rng.integers(0, cols)] = 0x7F80               # one infinity
    b[8, rng.integers(0, cols)] = 0xFF80
    b[9, rng.integers(0, cols)] = 0x7FC0               # one NaN
    b[10, rng.integers(0, cols)] = 0xFFFF
    return b


@pytest.mark.parametrize("cols", [1, 8, 15, 16, 17, 100, 128, 1003, 4096])
def test_save8_and_restore8(cuda, cols):
    """Codes, exponents and restored values are the definition's, bit for bit."""
    b = special_rows(cols, cols)
    rows = b.shape[0]
    saved = ql.alloc_saved8(rows, cols)
    full, back = out(rows, cols)
    ql.qlinear_save8(to_dev(b), rows, cols, saved)
    ql.qlinear_restore8(saved, rows, cols, back)
    assert ql.qlinear_sync_status() == ql.QL_OK
    codes, exps = R.save8(bf16_to_f64(b))
    assert np.array_equal(saved[1].cpu().numpy(), exps)
    assert np.array_equal(saved[0].cpu().numpy(), codes)
    ref = R.restore8(codes, exps, cols)
    got = f64(back)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(got[~np.isnan(ref)], ref[~np.isnan(ref)])
    assert untouched(full, rows, cols)


@pytest.mark.parametrize("fmt,M,F,K", [("int4", 1, 33, 256), ("int4", 32, 100, 512), ("int6", 40, 1003, 256),
                                       ("affine", 300, 130, 512), ("int4", 300, 9700, 256)])
def test_gated_checkpoint(cuda, fmt, M, F, K):
    """The saved g and u are within half a step of the accumulators, themselves within 1e-2 rms of exact; the
    scale is no coarser than the values need (its top code has seven bits); padding columns hold zeros."""
    bits, group = (4, 64) if fmt == "affine" else (0, 0)
    L = layer(fmt, 2 * F, K, 21, bits, group)
    xb = scaled_x(L, M, 22)
    h, saved = run_gated(L, xb, M, "silu", save=True)
    gu = (bf16_to_f64(xb) @ L.wref.T).reshape(2 * M, F)
    codes, exps = saved[0].cpu().numpy(), saved[1].cpu().numpy()
    check_h(f64(h), gu[0::2], gu[1::2], "silu", "h beside the checkpoint")
    step = np.repeat(np.ldexp(1.0, exps.astype(int) - 127), 16, axis=1)[:, :F]
    got = R.restore8(codes, exps, F)
    assert np.all(np.abs(got - gu) <= 0.5 * step + 1e-2 * max(2.0, rms(gu)))
    top = np.abs(codes.reshape(2 * M, -1, 16).astype(int)).max(-1)
    assert top.max() <= 127 and top.min() >= 64
    assert np.all(codes[:, F:] == 0)
    back = torch.empty((2 * M, F), dtype=torch.bfloat16, device="cuda")
    ql.qlinear_restore8(saved, 2 * M, F, back)
    assert np.array_equal(f64(back), got)


# More tiles than SMs, two tiles of tokens: a CTA finishes several tiles, alone from its scratch tile (long K) or with the
# dequantisers' help (short K: one stage a tile, fewer stages than the ring, an odd number of them; with and without a
# checkpoint the two meet at different K)
@pytest.mark.parametrize("save", [False, True])
@pytest.mark.parametrize("fmt,bits,group,K", [("affine", 4, 64, 64), ("affine", 8, 64, 192), ("affine", 2, 64, 320),
                                              ("int6", 0, 0, 512), ("int4", 0, 0, 2048), ("int4", 0, 0, 2304),
                                              ("int6p", 0, 0, 4352)])
def test_gated_many_tiles(cuda, fmt, bits, group, K, save):
    M, F = 270, 5010
    L = layer(fmt, 2 * F, K, K, bits, group)
    xb = scaled_x(L, M, K + 1)
    h, saved = run_gated(L, xb, M, "silu", save)
    gu = bf16_to_f64(xb) @ L.wref.T
    check_h(f64(h), gu[:, :F], gu[:, F:], "silu", f"{fmt} K={K}")
    again, saved2 = run_gated(L, xb, M, "silu", save)
    assert torch.equal(h, again)
    if save:
        assert torch.equal(saved[0], saved2[0]) and torch.equal(saved[1], saved2[1])
        gu = gu.reshape(2 * M, F)
        exps = saved[1].cpu().numpy()
        step = np.repeat(np.ldexp(1.0, exps.astype(int) - 127), 16, axis=1)[:, :F]
        got = R.restore8(saved[0].cpu().numpy(), exps, F)
        assert np.all(np.abs(got - gu) <= 0.5 * step + 1e-2 * max(2.0, rms(gu)))


# ---- backward ----------------------------------------------------------------------------------------------

SHAPES = [(1, 34, 256), (5, 200, 512), (32, 2006, 768), (33, 66, 512), (77, 130, 1280), (300, 1000, 512)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("fmt,bits,group", FORMATS)
def test_gemm_dx(cuda, fmt, bits, group, M, N, K):
    L = layer(fmt, N, K, 31, bits, group)
    yb = bf16(np.random.default_rng(32).normal(size=(M, N)) * 1e-3)
    full, dx = out(M, K)
    ql.qlinear_gemm_dx(L.desc, *L.packed(), to_dev(yb), M, dx)
    assert ql.qlinear_sync_status() == ql.QL_OK
    check_dx(f64(dx), bf16_to_f64(yb), L.wref, f"{fmt}{bits} M={M} N={N} K={K}")
    assert untouched(full, M, K)


@pytest.mark.parametrize("fmt,bits,group,M,N,K", [
    ("int4", 0, 0, 2100, 128, 2304),    # a whole wave of tiles and some split ones
    ("int4", 0, 0, 40, 64, 256 * 74),   # 148 tiles: whole waves only
    ("int4", 0, 0, 3, 1, 256), ("int4", 0, 0, 257, 63, 256), ("int6", 0, 0, 600, 333, 512),
    ("affine", 4, 32, 50, 77, 96), ("affine", 8, 64, 50, 77, 64), ("affine", 2, 32, 9, 77, 64),
    ("affine", 4, 32, 2, 9, 32), ("affine", 8, 128, 33, 77, 640), ("int4", 0, 0, 2, 27648, 256)])
def test_gemm_dx_odd_sizes(cuda, fmt, bits, group, M, N, K):
    L = layer(fmt, N, K, 33, bits, group)
    yb = bf16(np.random.default_rng(34).normal(size=(M, N)) * 1e-3)
    full, dx = out(M, K)
    ql.qlinear_gemm_dx(L.desc, *L.packed(), to_dev(yb), M, dx)
    assert ql.qlinear_sync_status() == ql.QL_OK
    check_dx(f64(dx), bf16_to_f64(yb), L.wref, f"{fmt}{bits} M={M} N={N} K={K}")
    assert untouched(full, M, K)


def test_gemm_dx_magnitudes(cuda):
    """Tokens and weight rows of very unlike magnitude: each token is held to its own rms."""
    N, K, M = 300, 512, 40
    L = layer("int4", N, K, 35)
    rng = np.random.default_rng(36)
    yb = bf16(rng.normal(size=(M, N)) * np.exp2(rng.integers(-60, 60, size=(M, 1)).astype(np.float64)))
    yb[7] = 0
    dx = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    ql.qlinear_gemm_dx(L.desc, *L.packed(), to_dev(yb), M, dx)
    assert ql.qlinear_sync_status() == ql.QL_OK
    got, ref = f64(dx), bf16_to_f64(yb) @ L.wref
    assert np.all(got[7] == 0)
    for m in range(M):
        if m != 7:
            close(got[m], ref[m], 1e-2 * rms(ref[m]) + half_ulp_bf16(ref[m]), f"token {m}")


def saved_of(gu, M, F):
    codes, exps = R.save8(gu.reshape(2 * M, F))
    v = R.restore8(codes, exps, F).reshape(M, 2, F)
    return (torch.from_numpy(codes).cuda(), torch.from_numpy(exps).cuda()), v[:, 0], v[:, 1]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("fmt,bits,group", FORMATS[:4])
def test_gated_backward(cuda, fmt, bits, group, M, N, K):
    """From a given checkpoint: dx, and (dg | du) to half a bf16 step plus the activations' fast forms (1e-5 of
    each factor's largest)."""
    F, kind = N // 2, R.ACTS[(M + N) % 3]
    L = layer(fmt, N, K, 41, bits, group)
    rng = np.random.default_rng(42)
    saved, g, u = saved_of(rng.normal(size=(M, 2, F)) * 2.0, M, F)
    hb = bf16(rng.normal(size=(M, F)) * 1e-3)
    dh = bf16_to_f64(hb)
    full, dx = out(M, K)
    gfull, dgu = out(M, N)
    ql.qlinear_gated_backward(L.desc, *L.packed(), saved, to_dev(hb), M, kind, dx, dgu=dgu)
    assert ql.qlinear_sync_status() == ql.QL_OK
    d = R.gated_backward(g, u, dh, kind)
    size = np.concatenate((np.abs(dh * u), np.abs(dh * g)), 1)
    assert np.all(np.abs(f64(dgu) - d) <= half_ulp_bf16(d) * (1 + 1e-3) + 1e-5 * size)
    check_dx(f64(dx), d, L.wref, f"{fmt}{bits} M={M}")
    assert untouched(full, M, K) and untouched(gfull, M, N)
    again = torch.empty_like(dx)
    ql.qlinear_gated_backward(L.desc, *L.packed(), saved, to_dev(hb), M, kind, again)
    assert torch.equal(again, dx)  # the same without the optional output, and from call to call


@pytest.mark.parametrize("kind", R.ACTS)
def test_activation_ranges(cuda, kind):
    """Large and tiny g: the value and the slope stay finite and right (F = 1: the group holds one value)."""
    g = np.array([0.0, 1e-30, -1e-30, 1e-3, -1e-3, 1.0, -1.0, 5.5, -5.5, 20.0, -20.0, 90.0, -90.0, 1e4, -1e4, 1e30,
                  -1e30])
    M = g.size
    L = layer("int4", 2, 256, 43)
    saved, gr, ur = saved_of(np.stack((g, np.ones(M)), 1).reshape(M, 2, 1), M, 1)
    hb = bf16(np.ones((M, 1)))
    dgu = torch.empty((M, 2), dtype=torch.bfloat16, device="cuda")
    dx = torch.empty((M, 256), dtype=torch.bfloat16, device="cuda")
    ql.qlinear_gated_backward(L.desc, *L.packed(), saved, to_dev(hb), M, kind, dx, dgu=dgu)
    assert ql.qlinear_sync_status() == ql.QL_OK
    with np.errstate(over="ignore", invalid="ignore"):
        small = R.gated_backward(np.clip(gr, -1e4, 1e4), ur, np.ones((M, 1)), kind)
    small[:, 1:] = np.where(np.abs(gr) > 1e4, np.maximum(gr, 0.0), small[:, 1:])
    # 1e-5: the fast exponential's error where act passes through its exponential tail
    assert np.all(np.abs(f64(dgu) - small) <= half_ulp_bf16(small) * (1 + 1e-3) + 1e-5 * np.maximum(1, np.abs(small)))


# ---- together ----------------------------------------------------------------------------------------------

class Block:
    """A gated block with its down projection, as a user's program holds it."""

    def __init__(self, fmt, F, K, seed, bits=0, group=0):
        self.up, self.down = layer(fmt, 2 * F, K, seed, bits, group), layer(fmt, K, F, seed + 1, bits, group)
        self.F, self.K = F, K

    def buffers(self, M):
        bf = lambda r, c: torch.zeros((r, c), dtype=torch.bfloat16, device="cuda")  # noqa: E731
        return dict(h=bf(M, self.F), y=bf(M, self.K), dh=bf(M, self.F), dx=bf(M, self.K),
                    saved=ql.alloc_saved8(2 * M, self.F), ws=ql.alloc_gated_workspace(self.up.desc, M),
                    ws_y=ql.alloc_gemm_workspace(self.down.desc, M),
                    ws_dh=ql.alloc_gemm_dx_workspace(self.down.desc, M),
                    ws_dx=ql.alloc_gemm_dx_workspace(self.up.desc, M))

    def step(self, x, dy, M, b, stream=None):
        u, d = self.up, self.down
        ql.qlinear_gated(u.desc, *u.packed(), x, M, "silu", b["h"], saved=b["saved"], workspace=b["ws"], stream=stream)
        ql.qlinear_gemm(d.desc, *d.packed(), b["h"], M, b["y"], workspace=b["ws_y"], stream=stream)
        ql.qlinear_gemm_dx(d.desc, *d.packed(), dy, M, b["dh"], workspace=b["ws_dh"], stream=stream)
        ql.qlinear_gated_backward(u.desc, *u.packed(), b["saved"], b["dh"], M, "silu", b["dx"], workspace=b["ws_dx"],
                                  stream=stream)


def test_block_forward_and_backward(cuda):
    """A whole block: y from x, dx from dy.  The chain's roundings (bf16 h and dh, 8-bit g and u: half a step of
    2^-6 to 2^-7 of a group's largest value, about 1.2e-2 of the rms at worst and 0.6e-2 on average) stay below
    3e-2 of the gradient's norm, and below 1e-2 of the output's, which meets no 8-bit value."""
    M, F, K = 150, 768, 512
    B = Block("int4", F, K, 51)
    xb = scaled_x(B.up, M, 52)
    dyb = bf16(np.random.default_rng(53).normal(size=(M, K)) * 1e-2)
    b = B.buffers(M)
    B.step(to_dev(xb), to_dev(dyb), M, b)
    assert ql.qlinear_sync_status() == ql.QL_OK
    gu = bf16_to_f64(xb) @ B.up.wref.T
    g, u = gu[:, :F], gu[:, F:]
    y = (R.act(g, "silu")[0] * u) @ B.down.wref.T
    dx = R.gated_backward(g, u, bf16_to_f64(dyb) @ B.down.wref, "silu") @ B.up.wref
    assert np.linalg.norm(f64(b["y"]) - y) <= 1e-2 * np.linalg.norm(y)
    assert np.linalg.norm(f64(b["dx"]) - dx) <= 3e-2 * np.linalg.norm(dx)


@pytest.mark.parametrize("M", [20, 150])
def test_captured_steps(cuda, M):
    """Two steps captured in graphs and replayed in turn give what eager calls give, with the inputs of the
    moment; they keep their own workspaces."""
    B = Block("int6", 256, 512, 61)
    rng = np.random.default_rng(62)
    xs = [to_dev(scaled_x(B.up, M, 63 + i)) for i in range(4)]
    dys = [to_dev(bf16(rng.normal(size=(M, 512)) * 1e-2)) for _ in range(4)]
    want = []
    for x, dy in zip(xs, dys):
        b = B.buffers(M)
        B.step(x, dy, M, b)
        want.append((b["y"], b["dx"], b["saved"][0]))
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        x, dy, b = xs[i].clone(), dys[i].clone(), B.buffers(M)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            B.step(x, dy, M, b)
        graphs.append((g, x, dy, b))
    for first in (0, 2):
        for i, (g, x, dy, b) in enumerate(graphs):
            x.copy_(xs[first + i])
            dy.copy_(dys[first + i])
            g.replay()
        torch.cuda.synchronize()
        for i, (_, _, _, b) in enumerate(graphs):
            y, dx, codes = want[first + i]
            assert torch.equal(b["y"], y) and torch.equal(b["dx"], dx) and torch.equal(b["saved"][0], codes)
    assert ql.qlinear_sync_status() == ql.QL_OK


def test_steps_on_two_streams(cuda):
    """Two streams, each with its own buffers and workspaces (one allocated by the call), at once."""
    M = 60
    B = Block("int4", 256, 512, 71)
    x = [to_dev(scaled_x(B.up, M, 72 + i)) for i in range(2)]
    dy = to_dev(bf16(np.random.default_rng(74).normal(size=(M, 512)) * 1e-2))
    want = []
    for i in range(2):
        b = B.buffers(M)
        B.step(x[i], dy, M, b)
        want.append(b)
    torch.cuda.synchronize()
    got, streams = [B.buffers(M) for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    got[1].update(ws=None, ws_dh=None, ws_dx=None)
    torch.cuda.synchronize()
    for _ in range(3):
        for i in range(2):
            B.step(x[i], dy, M, got[i], stream=streams[i])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for k in ("h", "y", "dh", "dx"):
            assert torch.equal(a[k], b[k]), k


def test_a_token_that_is_not_finite_spoils_only_itself(cuda):
    M, F, K = 50, 200, 512
    L = layer("int4", 2 * F, K, 81)
    xb = scaled_x(L, M, 82)
    clean, saved0 = run_gated(L, xb, M, "silu", save=True)
    xb[9, 3] = 0x7F80
    xb[30, 5] = 0x7FC0
    h, saved = run_gated(L, xb, M, "silu", save=True)
    rest = [m for m in range(M) if m not in (9, 30)]
    assert torch.equal(h[rest], clean[rest])
    assert bool(torch.isnan(h[30]).all())
    e = saved[1].view(M, 2, -1)
    assert bool((e[30] == 255).all()) and bool((e[rest] != 255).all())
    hb = to_dev(bf16(np.random.default_rng(83).normal(size=(M, F))))
    dx0, dx = (torch.empty((M, K), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ql.qlinear_gated_backward(L.desc, *L.packed(), saved0, hb, M, "silu", dx0)
    ql.qlinear_gated_backward(L.desc, *L.packed(), saved, hb, M, "silu", dx)
    assert ql.qlinear_sync_status() == ql.QL_OK
    assert torch.equal(dx[rest], dx0[rest]) and bool(torch.isnan(dx[30]).all())


@pytest.mark.parametrize("fmt,M", [("int4", 1), ("int4", 4), ("int6", 2), ("affine", 16), ("int4", 20), ("int4", 300)])
def test_gated_wait_runs_out_then_recovers(cuda, fmt, M):
    """The give-up path of the bounded waits (copies withheld on purpose), as tests/test_gpu_timeout drives it."""
    bits, group = (4, 64) if fmt == "affine" else (0, 0)
    L = layer(fmt, 2048, 512, 91, bits, group)
    xb = scaled_x(L, M, 92)
    h = torch.empty((M, 1024), dtype=torch.bfloat16, device="cuda")
    assert ql.qlinear_sync_status() == ql.QL_OK
    ql.qlinear_set_withhold_copies(True)
    try:
        ql.qlinear_gated(L.desc, *L.packed(), to_dev(xb), M, "silu", h)
        status = ql.qlinear_sync_status()
    finally:
        ql.qlinear_set_withhold_copies(False)
    assert status == ql.QL_ERR_TIMEOUT
    h, _ = run_gated(L, xb, M, "silu")
    gu = bf16_to_f64(xb) @ L.wref.T
    check_h(f64(h), gu[:, :1024], gu[:, 1024:], "silu", "after a time-out")


@pytest.mark.parametrize("M", [4, 300])
def test_dx_wait_runs_out_then_recovers(cuda, M):
    L = layer("int4", 512, 1024, 93)
    yb = bf16(np.random.default_rng(94).normal(size=(M, 512)))
    dx = torch.empty((M, 1024), dtype=torch.bfloat16, device="cuda")
    assert ql.qlinear_sync_status() == ql.QL_OK
    ql.qlinear_set_withhold_copies(True)
    try:
        ql.qlinear_gemm_dx(L.desc, *L.packed(), to_dev(yb), M, dx)
        status = ql.qlinear_sync_status()
    finally:
        ql.qlinear_set_withhold_copies(False)
    assert status == ql.QL_ERR_TIMEOUT
    ql.qlinear_gemm_dx(L.desc, *L.packed(), to_dev(yb), M, dx)
    assert ql.qlinear_sync_status() == ql.QL_OK
    check_dx(f64(dx), bf16_to_f64(yb), L.wref, "after a time-out")


def test_binding_refusals_on_the_gpu(cuda):
    L = layer("int4", 64, 256, 95)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    saved = ql.alloc_saved8(4, 32)
    ok = dict(x=bf(2, 256), h=bf(2, 32), saved=saved, workspace=None)
    for k, v, want in (("x", bf(2, 256).float(), ql.QL_ERR_SHAPE), ("x", bf(1, 256), ql.QL_ERR_SHAPE),
                       ("x", bf(256, 4).t(), ql.QL_ERR_SHAPE), ("h", bf(2, 31), ql.QL_ERR_SHAPE),
                       ("h", bf(2, 32).cpu(), ql.QL_ERR_UNSUPPORTED),
                       ("saved", ql.alloc_saved8(3, 32), ql.QL_ERR_SHAPE),
                       ("saved", (saved[0].float(), saved[1]), ql.QL_ERR_SHAPE),
                       ("workspace", torch.empty(256, dtype=torch.uint8, device="cuda"), ql.QL_ERR_SHAPE)):
        a = {**ok, k: v}
        with pytest.raises(ql.QLinearError) as e:
            ql.qlinear_gated(L.desc, *L.packed(), a["x"], 2, "silu", a["h"], saved=a["saved"], workspace=a["workspace"])
        assert e.value.status == want, k
    with pytest.raises(ql.QLinearError) as e:
        ql.qlinear_gemm_dx(L.desc, L.codes[:-16], L.gmeta, L.steps, bf(2, 64), 2, bf(2, 256))
    assert e.value.status == ql.QL_ERR_SHAPE
    assert ql.qlinear_sync_status() == ql.QL_OK
