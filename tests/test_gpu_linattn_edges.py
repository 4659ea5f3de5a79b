"""Edges of the linear attention with a fixed decay for each head: large states that fade, waits, refusals, NaN."""
import warnings

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


def calls(T, H, d, n, seed):
    q, k, v, do, S0, dST = make(n * T, H, d, torch.bfloat16, n, seed=seed)
    g = torch.full((H,), -0.05, device="cuda")

    def both(flags=None):
        """(o, ST) and (dq, dk, dv, dS0)"""
        return (pace.pace_linattn_forward(q, k, v, g, num_seqs=n, S0=S0, flags=flags),
                pace.pace_linattn_backward(q, k, v, g, do, num_seqs=n, S0=S0, dST=dST, flags=flags))

    return both


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [1, 64, 200, 4000])
def test_a_wait_that_runs_out_is_seen(T, d, waits):
    """The first barrier never completes: the launch ends, sets the flag, and leaves NaN where its results were to be, with
    a flag word or without; the calls after it are right.  (4000 tokens are cut into stretches.)"""
    both = calls(T, 1, d, 1, 23)
    want = both()
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    waits(100, 16)
    a.record()
    (o, ST), (dq, dk, dv, dS0) = both(flags)
    b.record()
    torch.cuda.synchronize()
    assert int(flags) == pace.PACE_FLAG_TIMEOUT
    assert a.elapsed_time(b) < 200.0                         # not the default limit of 2 s a wait
    # the first block of a backward pass walks for dv and dS0, of cut sequences over the first rows
    for x in (o, ST, dv[:200], dS0):
        assert bool(torch.isnan(x).all())
    (o, ST), (_, _, dv, dS0) = both()
    assert all(bool(torch.isnan(x).all()) for x in (o, ST, dv[:200], dS0))
    waits(0, 0)
    flags.zero_()
    got = both(flags)
    assert int(flags) == 0
    assert all(torch.equal(x, y) for w, r in zip(want, got) for x, y in zip(w, r))


def test_a_wait_that_runs_out_is_one_blocks(waits):
    """200 sequences of one head on 148 blocks: the first block's two sequences are NaN, the others what they were."""
    n, T, d = 200, 70, 128
    (o, ST), _ = want = calls(T, 1, d, n, 24)()
    waits(100, 16)
    (o2, ST2), _ = calls(T, 1, d, n, 24)()
    lost = torch.zeros(n, dtype=torch.bool, device="cuda")
    lost[[0, 148]] = True
    o, o2 = o.view(n, T, d), o2.view(n, T, d)
    assert torch.equal(o[~lost], o2[~lost]) and torch.equal(ST[~lost], ST2[~lost])
    assert bool(torch.isnan(o2[lost]).all()) and bool(torch.isnan(ST2[lost]).all())


def test_what_is_missing_is_refused():
    q, k, v, do, S0, _ = make(8, 2, 64, torch.bfloat16, 8)
    for call in (lambda: pace.pace_linattn_forward(q, k, v, None),
                 lambda: pace.pace_linattn_backward(q, k, v, None, do),
                 lambda: pace.pace_linattn_step(S0, q, k, v, None),
                 lambda: pace.pace_linattn_step(None, q, k, v, torch.zeros(2, device="cuda")),
                 lambda: pace.pace_linattn_forward(q, k, v, torch.zeros(2, device="cuda"), workspace=0)):
        with pytest.raises(ValueError):
            call()


def test_detached_outputs_are_announced():
    """Nothing is recorded for autograd: a call that would be expected to is told so, one in an autograd function or
    without gradients is not, and the values are the same."""
    q, k, v, do, S0, _ = make(8, 2, 64, torch.float32, 8)
    g, w = torch.tensor([-0.1, -0.2], device="cuda"), torch.ones(64, device="cuda")
    want = pace.pace_linattn_forward(q, k, v, g, S0=S0[:1])[0]

    def all_of():
        return [lambda: pace.pace_linattn_forward(q, k, v, g, S0=S0[:1])[0],
                lambda: pace.pace_linattn_backward(q, k, v, g, do, S0=S0[:1])[0],
                lambda: pace.pace_linattn_step(S0.clone(), q, k, v, g),
                lambda: pace.pace_qk_norm_rotate(q, k, w, w)[0],
                lambda: pace.pace_qk_norm_rotate_backward(q, k, w, w, None, None, do, do)[0]]

    with warnings.catch_warnings():
        warnings.simplefilter("error")
        for call in all_of():
            call()
        q.requires_grad_()
        with torch.no_grad():
            for call in all_of():
                call()
    for call in all_of():
        with pytest.warns(UserWarning, match="detached"):
            assert not call().requires_grad
    with pytest.warns(UserWarning):
        assert torch.equal(want, pace.pace_linattn_forward(q, k, v, g, S0=S0[:1])[0])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")], ids=str)
def test_what_is_not_a_number_stays_causal(what, d, dt):
    """A NaN or infinity at token t, in one channel or all of them, reaches the outputs from t on (gradients for k and v: up
    to t) and none that the formulas keep from it, which come out bit for bit as without it.  (bf16 with d = 64 and 128:
    but for the other tokens of its 64, counted from the sequence's first one.)"""
    dt, H, T = DT[dt], 2, 150
    cu, dev_cu = lengths(70, 80)
    base = dict(zip(("q", "k", "v", "do"), make(T, H, d, dt, 2, seed=31)[:4]))
    S0, dST = make(T, H, d, dt, 2, seed=32)[4:]
    g = torch.tensor([-0.02, -0.3], device="cuda")

    def run(x, states):
        s = dict(S0=S0) if states else {}
        o, ST = pace.pace_linattn_forward(x["q"], x["k"], x["v"], g, cu_seqlens=dev_cu, max_len=80, **s)
        if states:
            s["dST"] = dST
        dq, dk, dv, _ = pace.pace_linattn_backward(x["q"], x["k"], x["v"], g, x["do"], cu_seqlens=dev_cu, max_len=80, **s)
        return dict(o=o, dq=dq, dk=dk, dv=dv)

    # which outputs an input reaches: from it on, up to it, at it alone
    on, upto, at = "on", "upto", "at"
    reach = dict(q=dict(o=at, dk=upto, dv=upto), k=dict(o=on, dq=on, dv=at), v=dict(o=on, dq=on, dk=at),
                 do=dict(dq=at, dk=upto, dv=upto))
    for states in (True, False):
        want = run(base, states)
        for name in reach:
            for t in (0, 5, 31, 63, 64, 69, 70, 100, 133, 134, 149):
                b, e = (0, 70) if t < 70 else (70, 150)
                for channels in (slice(None), slice(d - 3, d - 2)):
                    x = dict(base, **{name: base[name].clone()})
                    x[name][t, 1, channels] = what
                    got = run(x, states)
                    for out, y in got.items():
                        hit = torch.zeros(T, H, dtype=torch.bool, device="cuda")
                        kind = reach[name].get(out)
                        first, last = t, t + 1
                        if dt == torch.bfloat16 and d > 32:
                            first = b + (t - b) // 64 * 64
                            last = min(first + 64, e)
                        if kind == on:
                            hit[first:e, 1] = True
                        elif kind == upto:
                            hit[b:last, 1] = True
                        elif kind == at:
                            hit[t, 1] = True
                        assert torch.equal(y[~hit], want[out][~hit]), (name, t, out, kind)
                        assert kind is None or not bool(torch.isfinite(y[t, 1]).all()), (name, t, out, kind)
