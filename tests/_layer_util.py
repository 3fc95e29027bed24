"""Inputs and error bounds shared by the layer operators' GPU tests.

Every bound is |got - ref| <= half |ref| + gamma mag: `half` is half a step of the output's type
relative to the value (2^-8 for bf16, 2^-24 for float32; the one rounding of the output), `mag` the
oracle's sum of absolute values, and gamma = c 2^-24 counts the float32 roundings on the longest way
from an input to the output."""
import numpy as np
import torch

from oracle import layer  # noqa: F401

U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def rnd(seed):
    return np.random.default_rng(seed)


def dev(a, dtype=F32):
    """Device tensor of a numpy array, rounded to dtype, and the exact values it holds."""
    if a is None:
        return None, None
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(dtype)
    return t.cuda(), t.double().numpy()


def both(values, dtype, params=()):
    """Device and exact numpy copies of a dict; names in `params` stay float32."""
    on, ref = {}, {}
    for k, v in values.items():
        on[k], ref[k] = dev(v, F32 if k in params else dtype)
    return on, ref


def cu_of(lens):
    return None if lens is None else np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def cu_dev(cu):
    return None if cu is None else torch.from_numpy(np.asarray(cu, np.int32)).cuda()


def check(name, got, ref, mag, gamma):
    assert (got is None) == (ref is None), name
    if got is None:
        return
    half = torch.finfo(got.dtype).eps / 2
    g = got.double().cpu().numpy()
    rows = ~np.isnan(ref)
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    assert np.isfinite(g[rows]).all(), f"{name}: non-finite values"
    err = np.abs(g - ref)[rows]
    bound = (half * np.abs(ref) + gamma * (1 + half) * mag)[rows] + 1e-37
    if err.size == 0:
        return
    worst = float((err / bound).max())
    print(f"{name}: worst {worst:.3f} of the bound (gamma {gamma:.1e})", flush=True)
    assert worst <= 1.0, f"{name}: {worst:.3f} of the bound"


# --- gamma, counted ------------------------------------------------------------------------------

def conv_gamma(W, pmax):
    # W + 1 roundings of p (SiLU's slope <= 1.1); the sigmoid: exponent's argument 2 |p|, exponential 2,
    # sum 1, reciprocal 2; product 1
    return U * (2 * W + 10 + 2 * pmax)


def conv_bwd_gamma(W, pmax, adds):
    # dp: twice the sigmoid's count and four products; dx: W more; parameter sums: one per addition
    return U * (4 * W + 24 + 4 * pmax + adds)


def scan_gamma(steps, umax, adds=0, ways=1):
    """A step size: 20 roundings and the argument's 2 |u|. A decay of exponent X: 3, and X times the
    step size's count and its own 4; over a path, sum X e^-X <= (2 / e) e^(-X/2), which the magnitude
    taken with A / 2 covers. Per step 3 more; 40 for the gate and the sum over 64 states."""
    return U * (ways * (3 * steps + 0.74 * (24 + 2 * umax)) + 40 + adds)


def half_A(ref):
    return {**ref, "A": ref["A"] / 2}


def norm_gamma(adds=0, backward=False):
    # a row sum: at most 38 additions, so 24 for its root, and 4; each part one to eight more. The
    # residual does not cancel the block's output in these tests: r keeps at least a fifth of its terms.
    return U * ((400 if backward else 200) + adds)
