"""How near the products grouped by expert are held to their definition in 64
bits: every element, and the whole result's norm."""
import experts_ref as ref
from layer_ref import U, within


def roundings(path, silu=False, combine=False):
    """Roundings to 16 bits that a result's relative error may add up to. Of the
    result: 1. On the tensor cores' path also the weights': activations of either
    sign at random give a product whose error is to its value, in the mean of
    squares, as each weight's error to the weight: 1; with silu(gate) * up those
    of both factors, and gate's magnified by its slope: 3; combined, the
    products': 1. Each is at most u = eps / 2 of its value and 0.4 u in the mean,
    which leaves room for the fp32 sums and the sample."""
    return 1 + (0 if path == "decode" else 3 if silu else 2 if combine else 1)


def off(got, want):
    """Relative error of the whole."""
    return float((got.double() - want).norm() / want.norm())


def close(got, want, tol, path, silu=False, combine=False):
    within(got, want, tol)
    err, most = off(got, want), roundings(path, silu, combine) * U[got.dtype]
    assert err <= most, f"off by {err} of the norm, more than {most}"


def check(call, A, W, routing, path, dtype, silu=False, combine=False):
    """call(A, ...) against the definition with the weights W."""
    weight_error = 0.0 if path == "decode" else ref.WEIGHT_ERROR[dtype]
    y, tol = ref.products(A, W, routing.experts, weight_error)
    if silu:
        y, tol = ref.silu_mul(y, tol)
    if combine:
        y, tol = ref.combine(y, tol, routing.weights, routing.experts, 0.0 if path == "decode" else U[dtype])
    close(call(A, silu_mul=silu, combine=combine), y, tol, path, silu, combine)
