"""Edges of the linear attention with a fixed decay for each head: large states that fade, waits, refusals, NaN."""
import numpy as np
import pytest
import torch

import bit_recurrent_state_pace_b200 as pace
from tests.test_gpu_linattn import DT, check_backward, check_forward, make

pytestmark = pytest.mark.gpu


def lengths(*lens):
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    return cu, torch.from_numpy(cu.astype(np.int32)).cuda()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_large_states_fade(d, dt):
    """States of 1e6 that a chunk of 64 tokens takes down to between 1e-2 and 1e-9 of that: what is left of them is held
    to the tolerance of what is left, not of what was there."""
    dt, H = DT[dt], 6
    g = torch.tensor([-0.07, -0.011, -0.0107, -0.2, -0.23, -0.33], device="cuda")
    cu, dev_cu = lengths(64, 200, 1, 63)
    q, k, v, do, S0, dST = make(int(cu[-1]), H, d, dt, len(cu) - 1, seed=21)
    S0, dST = 1e6 * S0, 1e6 * dST
    o, ST = pace.pace_linattn_forward(q, k, v, g, cu_seqlens=dev_cu, max_len=200, S0=S0)
    check_forward(q, k, v, g, S0, cu, o, ST, dt)
    grads = pace.pace_linattn_backward(q, k, v, g, do, cu_seqlens=dev_cu, max_len=200, S0=S0, dST=dST)
    check_backward(q, k, v, g, S0, do, dST, cu, grads, dt)


@pytest.fixture
def waits():
    """pace_debug_linattn_wait, with the defaults back at the end."""
    yield pace.pace_debug_linattn_wait
    torch.cuda.synchronize()
    pace.pace_debug_linattn_wait(0, 0)


@pytest.mark.parametrize("d", [64, 128])
def test_a_wait_is_bounded_by_its_work(d, waits):
    """One sequence of 16384 chunks that nothing says is long (max_len = 1), so that it is walked as one item, with short
    ones behind it on the same block: its states are waited for as long as its chunks take (30 ms), however few tests (1 ms)
    one wait has; the result is that of the default limit."""
    T, H = 1 << 20, 1
    _, dev_cu = lengths(T, *[1] * 200)
    q, k, v, do, S0, dST = make(T + 200, H, d, torch.bfloat16, 201, seed=22)
    g = torch.tensor([-0.01], device="cuda")

    def both():
        flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = pace.pace_linattn_forward(q, k, v, g, cu_seqlens=dev_cu, max_len=1, S0=S0, flags=flags)
        out += pace.pace_linattn_backward(q, k, v, g, do, cu_seqlens=dev_cu, max_len=1, S0=S0, dST=dST, flags=flags)
        return out, int(flags)

    want, flags = both()
    assert flags == 0
    waits(100, 0)
    got, flags = both()
    assert flags == 0
    assert all(torch.equal(a, b) for a, b in zip(want, got))
