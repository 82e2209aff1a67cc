"""The gated block on layers whose groups and metadata differ much in magnitude (GPU only).

The tolerances are those of tests/test_gpu_gated: an accumulator within 1e-2 rms of exact, the norm of the error
of h within 4e-3.  A group whose weights are 2^r below the row's largest counts as much as the others here, since
the elements of x that meet it are 2^r larger; bf16 elements that far apart are exact in the GEMM's fp16 rows.
"""
import numpy as np
import pytest

from tests import edge_inputs as E
from tests import ffn_reference as R
from tests.gpu_helpers import Layer, bf16_to_f64, half_ulp_bf16
from tests.test_gpu_edge_cases import INT4_GEMM_BOUND_KINDS, edge_layer, int4_weight_error_bound
from tests.test_gpu_gated import FORMATS, MAX_SLOPE, bf16, check_h, f64, layer, rms, run_gated
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


# ---- metadata and activations at the edges of the formats ------------------------------------------------------

GEMV_KINDS = tuple(k for k in E.X_KINDS if k != "wide20")


@pytest.mark.parametrize("M", [1, 7, 20, 42, 210])
@pytest.mark.parametrize("fmt,bits,group", FORMATS)
def test_gated_edge_inputs(cuda, fmt, bits, group, M):
    """tests/edge_inputs through the block, each (weight category, activation kind) on its own rms: gate and up row
    of a feature have one category.  The decode forms take the kinds that the GEMVs take.  The int4 GEMM's bound for
    an outlier on a weight at its zero point (tests/test_gpu_edge_cases) is that of the block's g and u as well."""
    F, K = 150, 2048
    L, cats, names = edge_layer(fmt, 2 * F, K, bits, group, seed=15)
    w = L.oracle_w().astype(np.float64)
    decode = M <= (32 if fmt == "affine" and group < 128 else 8)
    kinds = GEMV_KINDS if decode else E.X_KINDS
    bad = []
    for turn in range(len(kinds) if M == 1 else 1):
        ks = [kinds[(m + turn) % len(kinds)] for m in range(M)]
        xb = E.activations(ks, K, seed=16 + turn)
        h, _ = run_gated(L, xb, M, "silu")
        h, gu = f64(h), bf16_to_f64(xb) @ w.T
        extra = int4_weight_error_bound(L.w, xb) if fmt == "int4" and not decode else np.zeros((M, 2 * F))
        for c, name in enumerate(names):
            sel = np.flatnonzero(cats[:F] == c)
            for kind in sorted(set(ks)):
                ms = [m for m in range(M) if ks[m] == kind]
                g, u = gu[np.ix_(ms, sel)], gu[np.ix_(ms, sel + F)]
                on = float(name == "zero slots" and kind in INT4_GEMM_BOUND_KINDS)
                eg = 1e-2 * rms(g) + 1e-3 + on * extra[np.ix_(ms, sel)]
                eu = 1e-2 * rms(u) + 1e-3 + on * extra[np.ix_(ms, sel + F)]
                a = R.act(g, "silu")[0]
                tol = np.abs(u) * MAX_SLOPE * eg + np.abs(a) * eu + MAX_SLOPE * eg * eu + half_ulp_bf16(a * u)
                err = np.abs(h[np.ix_(ms, sel)] - a * u)
                if not np.all(err <= tol):
                    bad.append(f"{name} x={kind}: {int((~(err <= tol)).sum())} of {err.size}, worst {np.nanmax(err / tol):.2f}")
    assert not bad, "\n".join(bad)


# ---- forms that few calls reach ---------------------------------------------------------------------------------

@pytest.mark.parametrize("fmt,bits,group", [("int6", 0, 0), ("int6p", 0, 0), ("affine", 2, 64), ("affine", 4, 64)])
def test_gated_32_token_tiles_two_a_sm(cuda, fmt, bits, group):
    """More tiles of 64 features than SMs at up to 32 tokens: two CTAs an SM, some of them with two tiles."""
    M, F, K = 20, 22000, 256
    L = layer(fmt, 2 * F, K, 220, bits, group)
    x = np.random.default_rng(221).normal(size=(M, K)) * 2.0 / (rms(L.wref) * np.sqrt(K))
    xb = bf16(x)
    h, saved = run_gated(L, xb, M, "gelu", True)
    gu = bf16_to_f64(xb) @ L.wref.T
    check_h(f64(h), gu[:, :F], gu[:, F:], "gelu", fmt)
    got = R.restore8(saved[0].cpu().numpy(), saved[1].cpu().numpy(), F)
    step = np.repeat(np.ldexp(1.0, saved[1].cpu().numpy().astype(int) - 127), 16, axis=1)[:, :F]
    assert np.all(np.abs(got - gu.reshape(2 * M, F)) <= 0.5 * step + 1e-2 * max(2.0, rms(gu)))
