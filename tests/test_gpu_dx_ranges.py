"""Input gradients of layers whose groups, rows and metadata differ much in magnitude, the dealing of split tiles,
and long rows of dy (GPU only).

A column of dx depends on that column of the weights alone, so small columns are held to their own rms: 1e-2 of it
for each value and 4e-3 for the norm of the error, the tolerances of tests/test_gpu_gated.
"""
import numpy as np
import pytest
import torch

import int6_quantized_linear_b200 as ql
from int6_quantized_linear_b200 import synth
from tests.gpu_helpers import Layer, bf16_to_f64, half_ulp_bf16
from tests.test_gpu_edge_cases import edge_layer
from tests.test_gpu_gated import FORMATS, bf16, check_dx, close, f64, layer, out, rms, saved_of, to_dev, untouched
from tests.test_gpu_gated_ranges import unlike_layer
from tests import ffn_reference as R

pytestmark = pytest.mark.gpu


def run_dx(L, yb, M):
    full, dx = out(M, L.K)
    ql.qlinear_gemm_dx(L.desc, *L.packed(), to_dev(yb), M, dx)
    assert ql.qlinear_sync_status() == ql.QL_OK
    assert untouched(full, M, L.K)
    return f64(dx)


def of_weights(fmt, N, K, w, bits=0, group=0):
    L = Layer(fmt, N, K, 0, bits, group, weights=w)
    L.wref = L.oracle_w().astype(np.float64)
    return L


# ---- magnitudes -------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("M", [5, 40, 300])
@pytest.mark.parametrize("r", [8, 14])
@pytest.mark.parametrize("fmt,bits,group", FORMATS)
def test_dx_columns_of_unlike_magnitude(cuda, fmt, bits, group, r, M):
    """The first 256 columns are 2^r times the others in every row."""
    N, K = 300, 768
    L = unlike_layer(fmt, bits, group, N, K, 300 + r, r)
    yb = bf16(np.random.default_rng(301).normal(size=(M, N)))
    got, ref = run_dx(L, yb, M), bf16_to_f64(yb) @ L.wref
    for name, c in (("large", slice(0, 256)), ("small", slice(256, K))):
        close(got[:, c], ref[:, c], 1e-2 * rms(ref[:, c]) + half_ulp_bf16(ref[:, c]), f"{fmt}{bits} {name} columns")


@pytest.mark.parametrize("M", [5, 300])
def test_dx_large_zero_step_that_no_group_uses(cuda, M):
    """int4 zero steps of 1000 with zero codes 0: the weights are q S, whatever the step."""
    N, K = 300, 768
    w = synth.int4_weights(310, N, K)
    w["zs"][:] = np.float16(1000.0).view(np.uint16)
    w["zc"][:] = 0
    L = of_weights("int4", N, K, w)
    yb = bf16(np.random.default_rng(311).normal(size=(M, N)))
    check_dx(run_dx(L, yb, M), bf16_to_f64(yb), L.wref, "unused zero step")


@pytest.mark.parametrize("M", [5, 300])
@pytest.mark.parametrize("fmt,bits,group", FORMATS)
def test_dx_rows_of_unlike_magnitude(cuda, fmt, bits, group, M):
    """Row steps over many powers of two (fp16 subnormals among them), dy the inverse, so that every row counts
    alike; and rows of zeros, whose dy is far above the others' and does not count."""
    N, K = 300, 512
    rng = np.random.default_rng(320)
    e = rng.integers(-8, 12, size=N) if fmt != "affine" else rng.integers(-60, 60, size=N)
    if fmt == "affine":
        w = synth.affine_weights(321, N, K, bits, group)
        for k in ("s", "b"):
            w[k] = (w[k].astype(np.int64) + (e[:, None] << 7)).astype(np.uint16)
            w[k][[7, 100]] = 0
    else:
        w = synth.int4_weights(321, N, K) if fmt == "int4" else synth.int6_weights(321, N, K)
        k = "ss" if fmt == "int4" else "st"
        v = w[k].view(np.float16).astype(np.float64) * 2.0 ** e[:, None]
        w[k] = v.astype(np.float16).view(np.uint16)
        w[k][[7, 100]] = 0
    L = of_weights(fmt, N, K, w, bits, group)
    assert not L.wref[[7, 100]].any()
    y = rng.normal(size=(M, N)) * 2.0 ** -e.astype(np.float64)
    y[:, [7, 100]] *= 2.0 ** 70
    yb = bf16(y)
    yb[M - 1, [7, 100]] = 0  # one token without them
    check_dx(run_dx(L, yb, M), bf16_to_f64(yb), L.wref, f"{fmt}{bits} rows")


@pytest.mark.parametrize("fmt,bits,group", FORMATS)
def test_dx_edge_inputs(cuda, fmt, bits, group):
    """tests/edge_inputs' weight categories: a token's dy is zero but for the rows of one category, and the token is
    held to its own rms.  dy is large enough for the smallest weights' gradients to be normal numbers."""
    N, K, M = 300, 2048, 42
    L, cats, names = edge_layer(fmt, N, K, bits, group, seed=25)
    w = L.oracle_w().astype(np.float64)
    y = np.random.default_rng(26).normal(size=(M, N)) * 2.0 ** 20
    y[cats[None, :] != (np.arange(M) % len(names))[:, None]] = 0
    yb = bf16(y)
    got, ref = run_dx(L, yb, M), bf16_to_f64(yb) @ w
    for m in range(M):
        close(got[m], ref[m], 1e-2 * rms(ref[m]) + half_ulp_bf16(ref[m]), f"{fmt}{bits} {names[m % len(names)]}")


# ---- the dealing of tiles ---------------------------------------------------------------------------------------

def dealing(M, N, K):
    """(tile class, whole waves, tiles of the rest, shares, shares that straddle two tiles, most pieces of a CTA), by
    the rule in csrc/gemm_dx.cuh."""
    c = 32 if M <= 32 else 64 if M <= 64 else 256
    tiles = -(-M // c)
    tokens = -(-(-(-M // tiles)) // 16) * 16
    ctas = min(148, torch.cuda.get_device_properties(0).multi_processor_count) * (1 if c == 256 else 2)
    all_tiles = -(-M // tokens) * -(-K // 128)
    steps = -(-N // 64)
    waves, rest = divmod(all_tiles, ctas)
    shares = max(rest, min(ctas, rest * steps // 8)) if rest else 0
    begin = [rest * steps * i // max(shares, 1) for i in range(shares + 1)]
    straddle = [(begin[i + 1] - 1) // steps > begin[i] // steps for i in range(shares)]
    return c, waves, rest, shares, sum(straddle), waves + (2 if any(straddle) else 1 if rest else 0)


# (M, N, K) of each tile class with split tiles alone and behind whole waves; the last has four pieces in a CTA, which
# takes the two accumulators of small tiles round twice
DEALS = [(300, 1250, 6400, 256, 0), (2100, 3000, 2304, 256, 1), (700, 700, 14336, 256, 2), (50, 1000, 25600, 64, 0),
         (50, 1400, 38400, 64, 1), (5, 1000, 25600, 32, 0), (5, 1400, 38400, 32, 1), (20, 600, 76800, 32, 2)]


@pytest.mark.parametrize("M,N,K,tile,waves", DEALS)
def test_dx_split_tiles(cuda, M, N, K, tile, waves):
    c, w, rest, shares, straddle, pieces = dealing(M, N, K)
    assert (c, w) == (tile, waves) and rest < shares and shares % rest and straddle > 0, "sizes that the rule splits"
    assert waves < 2 or pieces == 4
    L = layer("int4", N, K, 330)
    yb = bf16(np.random.default_rng(331).normal(size=(M, N)) * 1e-3)
    got = run_dx(L, yb, M)
    check_dx(got, bf16_to_f64(yb), L.wref, f"M={M} N={N} K={K}")
    assert np.array_equal(got, run_dx(L, yb, M))


@pytest.mark.parametrize("M,K", [(40, 256 * 148), (20, 256 * 148), (1000, 4736)])
def test_dx_whole_waves_only(cuda, M, K):
    c, waves, rest, _, _, _ = dealing(M, 64, K)
    assert waves >= 1 and rest == 0
    L = layer("affine", 64, K, 332, 8, 64)
    yb = bf16(np.random.default_rng(333).normal(size=(M, 64)))
    check_dx(run_dx(L, yb, M), bf16_to_f64(yb), L.wref, f"M={M}")


# ---- long rows of dy --------------------------------------------------------------------------------------------

@pytest.mark.parametrize("N", [9001, 32768 + 8, 33333, 70000])
@pytest.mark.parametrize("M", [3, 70])
def test_dx_long_rows(cuda, N, M):
    """Rows of dy that more threads keep in registers, and rows that are read twice; with and without 16-byte rows."""
    K = 64
    L = layer("affine", N, K, 340, 4, 64)
    yb = bf16(np.random.default_rng(341).normal(size=(M, N)) * 1e-2)
    check_dx(run_dx(L, yb, M), bf16_to_f64(yb), L.wref, f"N={N}")


# ---- one workspace for many layers ------------------------------------------------------------------------------

@pytest.mark.parametrize("M", [4, 40, 300])
def test_calls_share_a_workspace(cuda, M):
    """Layers of unlike scales, one after the other on one stream with one workspace, eager and in a graph: each call
    gives what it gives with a workspace of its own."""
    F, K = 192, 512
    layers = []
    for i, e in enumerate((0, 6, -4, 9)):
        w = synth.int4_weights(370 + i, 2 * F, K)
        w["ss"] = (w["ss"].view(np.float16).astype(np.float64) * 2.0 ** e).astype(np.float16).view(np.uint16)
        layers.append(of_weights("int4", 2 * F, K, w))
    rng = np.random.default_rng(375)
    x, dy = to_dev(bf16(rng.normal(size=(M, K)) * 0.1)), to_dev(bf16(rng.normal(size=(M, 2 * F))))
    dh = to_dev(bf16(rng.normal(size=(M, F))))
    need = max(ql.qlinear_gated_workspace_bytes(layers[0].desc, M), ql.qlinear_gemm_dx_workspace_bytes(layers[0].desc, M))
    bf = lambda r, c: torch.empty((r, c), dtype=torch.bfloat16, device="cuda")  # noqa: E731

    def run(shared, o):
        for L, (h, saved, dx, dx2) in zip(layers, o):
            ql.qlinear_gated(L.desc, *L.packed(), x, M, "silu", h, saved=saved, workspace=shared)
            ql.qlinear_gemm_dx(L.desc, *L.packed(), dy, M, dx, workspace=shared)
            ql.qlinear_gated_backward(L.desc, *L.packed(), saved, dh, M, "silu", dx2, workspace=shared)

    outs = lambda: [(bf(M, F), ql.alloc_saved8(2 * M, F), bf(M, K), bf(M, K)) for _ in layers]  # noqa: E731
    want, eager, replayed = outs(), outs(), outs()
    for L, o in zip(layers, want):
        ql.qlinear_gated(L.desc, *L.packed(), x, M, "silu", o[0], saved=o[1])
        torch.cuda.synchronize()
        ql.qlinear_gemm_dx(L.desc, *L.packed(), dy, M, o[2])
        torch.cuda.synchronize()
        ql.qlinear_gated_backward(L.desc, *L.packed(), o[1], dh, M, "silu", o[3])
        torch.cuda.synchronize()
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for _ in range(5):
        run(ws, eager)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(ws, replayed)
    for _ in range(5):
        g.replay()
    assert ql.qlinear_sync_status() == ql.QL_OK
    for a in (eager, replayed):
        for p, q in zip(a, want):
            assert torch.equal(p[0], q[0]) and torch.equal(p[2], q[2]) and torch.equal(p[3], q[3])
            assert torch.equal(p[1][0], q[1][0]) and torch.equal(p[1][1], q[1][1])


# ---- the backward pass ------------------------------------------------------------------------------------------

@pytest.mark.parametrize("M,N,K", [(5, 200, 512), (33, 66, 512), (300, 1000, 512)])
@pytest.mark.parametrize("fmt,bits,group", FORMATS[4:])
def test_backward_of_the_other_formats(cuda, fmt, bits, group, M, N, K):
    F, kind = N // 2, R.ACTS[M % 3]
    L = layer(fmt, N, K, 350, bits, group)
    rng = np.random.default_rng(351)
    saved, g, u = saved_of(rng.normal(size=(M, 2, F)) * 2.0, M, F)
    hb = bf16(rng.normal(size=(M, F)) * 1e-3)
    full, dx = out(M, K)
    ql.qlinear_gated_backward(L.desc, *L.packed(), saved, to_dev(hb), M, kind, dx)
    assert ql.qlinear_sync_status() == ql.QL_OK
    check_dx(f64(dx), R.gated_backward(g, u, bf16_to_f64(hb), kind), L.wref, f"{fmt}{bits} M={M}")
    assert untouched(full, M, K)


@pytest.mark.parametrize("kind", R.ACTS)
def test_backward_of_large_values(cuda, kind):
    """g and u up to the largest that the 8-bit form holds (2^127), dh so that the gradients stay in range; and dh up
    to 2^120 with small u."""
    F, K = 64, 256
    L = layer("int4", 2 * F, K, 360)
    rng = np.random.default_rng(361)
    es = [20, 60, 90, 104, 105, 110, 118, 122, 126]
    v = rng.uniform(1.0, 1.9, size=(2 * len(es), 2, F)) * np.where(rng.random((2 * len(es), 2, F)) < 0.5, -1, 1)
    dh = rng.normal(size=(2 * len(es), F))
    for i, e in enumerate(es):
        v[i] *= 2.0 ** e
        dh[i] *= 2.0 ** -e
        v[len(es) + i] *= 2.0 ** -10
        dh[len(es) + i] *= 2.0 ** min(e, 120)
    M = 2 * len(es)
    saved, g, u = saved_of(v, M, F)
    hb = bf16(dh)
    dx = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    dgu = torch.empty((M, 2 * F), dtype=torch.bfloat16, device="cuda")
    ql.qlinear_gated_backward(L.desc, *L.packed(), saved, to_dev(hb), M, kind, dx, dgu=dgu)
    assert ql.qlinear_sync_status() == ql.QL_OK
    dh = bf16_to_f64(hb)
    d = R.gated_backward(np.clip(g, -1e4, 1e4), u, dh, kind)  # past 1e4 the slope is 0 or 1, and act is 0 or g
    d[:, F:] = np.where(g > 1e4, dh * g, np.where(g < -1e4, 0.0, d[:, F:]))
    got = f64(dgu)
    size = np.concatenate((np.abs(dh * u), np.abs(dh * g)), 1)
    assert np.all(np.abs(got - d) <= half_ulp_bf16(d) * (1 + 1e-3) + 1e-5 * size)
    gotx, ref = f64(dx), d @ L.wref
    for m in range(M):
        close(gotx[m], ref[m], 1e-2 * rms(ref[m]) + half_ulp_bf16(ref[m]), f"row {m}")
