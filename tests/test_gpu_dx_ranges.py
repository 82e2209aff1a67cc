"""Input gradients of layers whose groups, rows and metadata differ much in magnitude (GPU only).

A column of dx depends on that column of the weights alone, so small columns are held to their own rms: 1e-2 of it
for each value and 4e-3 for the norm of the error, the tolerances of tests/test_gpu_gated.
"""
import numpy as np
import pytest
import torch

import int6_quantized_linear_b200 as ql
from int6_quantized_linear_b200 import synth
from tests.gpu_helpers import Layer, bf16_to_f64, half_ulp_bf16
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
