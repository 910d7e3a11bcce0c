"""The bound that the few-row int4 products are held to tells exact codes from
rounded weights: a mistake planted in the oracle passes it nowhere."""
import numpy as np
import pytest

import a16w4_cases as C
import oracle


@pytest.mark.parametrize("M,N,K", [(1, 700, 256), (2, 1000, 64), (9, 300, 832), (16, 257, 4096)])
@pytest.mark.parametrize("fmt", ["f32", "asym"])
def test_rounded_weights_fail_the_bound_of_exact_codes(M, N, K, fmt):
    rng = np.random.default_rng(M + N)
    qw, sw, zw = C.weights(rng, N, K, fmt)
    if fmt == "asym":            # zeros that are no multiple of the scales
        zw = (zw * rng.uniform(0.9, 1.1, zw.shape)).astype(np.float32)
    x = C.integer_rows(rng, M, K).astype(np.float64)
    w = C.real(qw, sw, zw)
    ref = oracle.a16w4(x, w)
    tol = C.exact_codes_tolerance(x, qw, sw, zw, ref)
    C.assert_close(C.bf16_round(ref), ref, tol)
    planted = C.bf16_round(oracle.a16w4(x, C.bf16_round(w).astype(np.float64)))
    with pytest.raises(AssertionError):
        C.assert_close(planted, ref, tol)
