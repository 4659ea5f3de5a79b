"""Further refusals of the linear-attention and query/key-norm entry points, on the CPU: all are found on the host before
anything is launched."""
import ctypes

import pytest
import torch

import bit_recurrent_state_pace_b200 as pace


def test_debug_limits_of_the_chunk_kernel():
    for tries, extra in ((99, 0), (200001, 0), (100, 8), (100, 32), (1001, 16), (0, 16)):
        with pytest.raises(pace.PaceError) as e:
            pace.pace_debug_linattn_wait(tries, extra)
        assert e.value.status == pace.PACE_ERR_INVALID_ARG
    pace.pace_debug_linattn_wait(100, 0)
    pace.pace_debug_linattn_wait(0, 0)


# rows of 2 heads of d = 64 in bf16: 256 bytes; the addresses are never looked at
A = 0x100000
FAR = [A + (i << 20) for i in range(12)]


def lin(stride=0, **kw):
    a = dict(num_seqs=2, num_heads=2, d_k=64, d_v=64, io_dtype=0, total_tokens=20, max_len=10, q_stride=stride,
             k_stride=stride, v_stride=stride, o_stride=stride)
    a.update(kw)
    return ctypes.byref(pace._LinattnDesc(*[a[n] for n, _ in pace._LinattnDesc._fields_]))


def forward(desc, q, k, v, o, S0=None, ST=None):
    return pace.lib.pace_linattn_forward(desc, q, k, v, FAR[9], None, S0, o, ST, None, None, None)


def backward(desc, q, k, v, do, dq, dk, dv, S0=None, dST=None, dS0=None):
    return pace.lib.pace_linattn_backward(desc, q, k, v, FAR[9], None, S0, do, dST, dq, dk, dv, dS0, None, None, None)


def test_outputs_over_inputs():
    q, k, v, o, S0, ST, do, dq, dk = FAR[:9]
    for bad in (q, k, v, q + 16, k - 16, v + 19 * 256):                     # one byte of one row is enough
        assert forward(lin(), q, k, v, bad) == 1, hex(bad)
        if bad != v + 19 * 256:                                             # (a step has two rows)
            assert pace.lib.pace_linattn_step(lin(), S0, q, k, v, FAR[9], bad, None) == 1, hex(bad)
    # parts of rows three times as wide: at the same columns of another row, or half over them
    for bad in (q, q + 768, q + 128, q + 256 + 16):
        assert forward(lin(384), q, q + 256, q + 512, bad) == 1, hex(bad)
    # two strides: the first rows are looked for
    assert forward(lin(o_stride=512), q, k, v, q) == 1
    assert forward(lin(o_stride=512), q, k, v, k + 256) == 1
    # states: 4 of 64 x 64 fp32
    assert forward(lin(), q, k, v, o, S0, S0 + 16) == 1 and forward(lin(), q, k, v, o, S0, S0 - 16) == 1
    assert forward(lin(), q, k, v, o, S0, q) == 1 and forward(lin(), q, k, v, o, S0, o + 512) == 1
    g = [q, k, v, do, dq, dk, o]
    for i in range(4, 7):
        for j in [x for x in range(7) if x != i]:
            a = list(g)
            a[i] = g[j] + 32
            assert backward(lin(), *a) == 1, (i, j)
    for other in (S0, ST):
        assert backward(lin(), *g, S0=S0, dST=ST, dS0=other + 4096) == 1
    assert pace.lib.pace_linattn_step(lin(), q, q + 16, k, v, FAR[9], o, None) == 1


def norm(**kw):
    a = dict(num_tokens=5, num_q_heads=4, num_k_heads=2, head_dim=64, rotary_dim=0, interleaved=0, norm=1, io_dtype=0,
             eps=1e-6, q_scale=1.0, q_stride=0, k_stride=0, q_out_stride=0, k_out_stride=0)
    a.update(kw)
    return ctypes.byref(pace._QkNormDesc(*[a[n] for n, _ in pace._QkNormDesc._fields_]))


def test_norm_outputs_over_other_inputs():
    q, k, qo, ko, dyq, dyk, ws, w = FAR[:8]

    def fwd(q, k, qo, ko, **kw):
        return pace.lib.pace_qk_norm_rotate(norm(**kw), q, k, None, None, None, None, qo, ko, None)

    def bwd(dq, dk, dwq=None, dwk=None, **kw):
        return pace.lib.pace_qk_norm_rotate_backward(norm(**kw), q, k, None, None, None, None, dyq, dyk, dq, dk, dwq, dwk, ws, None)

    assert fwd(q, k, k, ko) == 1 and fwd(q, k, qo, q) == 1 and fwd(q, k, q + 16, ko) == 1 and fwd(q, k, qo, qo) == 1
    assert fwd(q, q, q, ko) == 1                                            # in place, but the other side reads it
    assert fwd(q, k, q, ko, q_out_stride=512) == 1
    assert bwd(k, dk=ko) == 1 and bwd(dyk, dk=ko) == 1 and bwd(q + 16, ko) == 1 and bwd(dyq + 512, ko) == 1
    assert bwd(qo, qo + 64) == 1 and bwd(qo, q) == 1 and bwd(qo, dyq) == 1
    assert bwd(dyq, ko, q_out_stride=512) == 1
    assert bwd(qo, ko, w, w) == 1 and bwd(qo, ko, w, w + 252) == 1


def test_the_binding_refuses_with_value_errors():
    q = torch.zeros(4, 2, 64)
    for name, call in (("norm", lambda: pace.pace_qk_norm_rotate(q, q, norm=["l2"])),
                       ("norm", lambda: pace.pace_qk_norm_rotate(q, q, norm={})),
                       ("norm", lambda: pace.pace_qk_norm_rotate_backward(q, q, None, None, None, None, q, q, norm=2)),
                       ("eps", lambda: pace.pace_qk_norm_rotate(q, q, eps=None)),
                       ("q_scale", lambda: pace.pace_qk_norm_rotate(q, q, q_scale="one")),
                       ("q_scale", lambda: pace.pace_qk_norm_rotate(q, q, q_scale=torch.ones(2)))):
        with pytest.raises(ValueError, match=name):
            call()
    with pytest.raises(ValueError, match="workspace"):
        pace._workspace("call", 256, [0], q, None)
