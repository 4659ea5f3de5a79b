"""How exact the linear attention is, in bounds that a lost part of a split operand does not pass."""
import numpy as np
import pytest
import torch

import bit_recurrent_state_pace_b200 as pace
from tests import operators_reference as ref
from tests.test_gpu_linattn import DT, close, f64, make, zeros

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [2, 17, 63, 64])
def test_scores_in_two_parts(T, d):
    """One sequence of one chunk and no state before it: outputs and gradients are P V alone.  P is two bf16 parts, so each
    term is off by 2^-16 (a rounding to 2^-8 of a rest that is at most 2^-8), and by the fp32 roundings; the result is
    rounded once."""
    H = 3
    q, k, v, do, _, _ = make(T, H, d, torch.bfloat16, 1, seed=41, states=False)
    g, cu = torch.tensor([-0.3, -0.01, 0.0], device="cuda"), [0, T]
    o, _ = pace.pace_linattn_forward(q, k, v, g)
    dq, dk, dv, _ = pace.pace_linattn_backward(q, k, v, g, do)
    S = zeros(1, H, d)
    wo, _, bo, _ = ref.forward(f64(q), f64(k), f64(v), f64(g), S, cu)
    want = [(wo, bo)] + list(ref.backward(f64(q), f64(k), f64(v), f64(g), S, f64(do), S, cu)[:3])
    for got, (w, b) in zip((o, dq, dk, dv), want):
        t = (2.0 ** -16 + ref.roundings32(T, d) * ref.U32) * b
        close(got, w, t + ref.UBF * (np.abs(w) + t))


def off(got, want):
    """The relative norm of the difference, for each head: the largest."""
    e = f64(got) - want
    axes = tuple(i for i in range(e.ndim) if i != 1)
    return float(np.sqrt((e * e).sum(axes) / (want * want).sum(axes)).max())


# One rounding to bf16 of numbers whose logarithms are spread evenly: 2^-8 / sqrt(3) * sqrt(3 / 8 / ln 2) = 1.66e-3 in the
# relative norm.  Outputs have one of their own and at most that of the state they are read from (the signs of queries and
# state are random, so the terms' errors add up as the terms do): sqrt(2) * 1.66e-3 = 2.35e-3.  A third, of a value or score
# left in one part, would make it sqrt(3) * 1.66e-3 = 2.9e-3.
BF16_OUT = 2.5e-3
# fp32 states in either type: 24 bits of every product, in a chunk at most 12 partial sums cut to 24 bits (2^-23 of them, one
# sided, half of that on average, of partial sums that are half of the whole on average: 3.6e-7), a decay within two units
# in the last place (1.2e-7), and two roundings a chunk that do not add up: below 1e-6.  Values cut to 16 bits would be off by
# 2^-17 = 7.6e-6 on average, rounded ones by 2^-17 at most.
STATE = 1e-6


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("n,T,H", [(1, 1500, 3), (60, 200, 3), (1, 3000, 1)])
def test_relative_norms(n, T, H, d, dt):
    """Heads that remember hundreds of tokens, in one piece and in stretches, with the states' gradient and without it."""
    dt = DT[dt]
    q, k, v, do, S0, dST = make(n * T, H, d, dt, n, seed=42)
    g, cu = torch.tensor([-0.002, -0.0005, -0.05][:H], device="cuda"), np.arange(n + 1) * T
    out = STATE if dt == torch.float32 else BF16_OUT
    for states in (True, False):
        s0, ds = (S0, dST) if states else (None, None)
        o, ST = pace.pace_linattn_forward(q, k, v, g, num_seqs=n, S0=s0)
        grads = pace.pace_linattn_backward(q, k, v, g, do, num_seqs=n, S0=s0, dST=ds)
        s64, d64 = (f64(S0), f64(dST)) if states else (zeros(n, H, d), zeros(n, H, d))
        wo, ws, _, _ = ref.forward(f64(q), f64(k), f64(v), f64(g), s64, cu)
        want = ref.backward(f64(q), f64(k), f64(v), f64(g), s64, f64(do), d64, cu)
        assert off(o, wo) <= out and off(ST, ws) <= STATE
        for got, (w, _) in zip(grads[:3], want[:3]):
            assert off(got, w) <= out
        if states:
            assert off(grads[3], want[3][0]) <= STATE
