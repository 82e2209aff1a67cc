"""The gated block on layers whose groups and metadata differ much in magnitude (GPU only).

The tolerances are those of tests/test_gpu_gated: an accumulator within 1e-2 rms of exact, the norm of the error
of h within 4e-3.  A group whose weights are 2^r below the row's largest counts as much as the others here, since
the elements of x that meet it are 2^r larger; bf16 elements that far apart are exact in the GEMM's fp16 rows.
"""
import numpy as np
import pytest

from tests import ffn_reference as R
from tests.gpu_helpers import Layer, bf16_to_f64
from tests.test_gpu_gated import FORMATS, bf16, check_h, f64, rms, run_gated
from int6_quantized_linear_b200 import synth

pytestmark = pytest.mark.gpu


def unlike_weights(fmt, bits, group, N, K, seed, r):
    """Weights whose first 256 columns are 2^r times the others'."""
    if fmt == "affine":
        w = synth.affine_weights(seed, N, K, bits, group)
        for k in ("s", "b"):
            w[k][:, :256 // group] += np.uint16(r << 7)  # bf16 exponents
    else:
        w = synth.int4_weights(seed, N, K) if fmt == "int4" else synth.int6_weights(seed, N, K)
        k = "ss" if fmt == "int4" else "st"
        w[k][:, :1] += np.uint16(r << 10)  # fp16 exponents (the steps are normal)
    return w


def unlike_layer(fmt, bits, group, N, K, seed, r):
    L = Layer(fmt, N, K, seed, bits, group, weights=unlike_weights(fmt, bits, group, N, K, seed, r))
    L.wref = L.oracle_w().astype(np.float64)
    return L


# 40 and 300 tokens: the GEMM's tiles of 32 and of 256 tokens; 4 tokens: with the checkpoint, on the GEMM
@pytest.mark.parametrize("M,save", [(4, True), (40, False), (300, True)])
@pytest.mark.parametrize("r", [8, 14])
@pytest.mark.parametrize("fmt,bits,group", FORMATS)
def test_gated_groups_of_unlike_magnitude(cuda, fmt, bits, group, r, M, save):
    F, K = 150, 1024
    L = unlike_layer(fmt, bits, group, 2 * F, K, 200 + r, r)
    x = np.random.default_rng(201).normal(size=(M, K)) * 2.0 / (rms(L.wref[:, 256:]) * np.sqrt(K))
    x[:, :256] *= 2.0 ** -r
    xb = bf16(x)
    h, saved = run_gated(L, xb, M, "silu", save)
    gu = bf16_to_f64(xb) @ L.wref.T
    assert 1.0 < rms(gu) < 4.0 and 0.3 < rms((bf16_to_f64(xb)[:, :256] @ L.wref[:, :256].T)) < 3.0
    check_h(f64(h), gu[:, :F], gu[:, F:], "silu", f"{fmt}{bits} groups 2^{r} apart")
    if save:
        exps = saved[1].cpu().numpy()
        step = np.repeat(np.ldexp(1.0, exps.astype(int) - 127), 16, axis=1)[:, :F]
        got = R.restore8(saved[0].cpu().numpy(), exps, F)
        assert np.all(np.abs(got - gu.reshape(2 * M, F)) <= 0.5 * step + 1e-2 * max(2.0, rms(gu)))
