"""Refusals of the linear-attention and query/key-norm entry points, and their workspace sizes, on the CPU: every
argument error is found on the host before anything is launched."""
import ctypes

import pytest
import torch

import bit_recurrent_state_pace_b200 as pace

# addresses that are never looked at: each call below is refused first
P, ODD, OFF4 = 0x10000, 0x10001, 0x10004


def lin(**kw):
    a = dict(num_seqs=2, num_heads=4, d_k=64, d_v=64, io_dtype=0, total_tokens=20, max_len=10, q_stride=0, k_stride=0,
             v_stride=0, o_stride=0)
    a.update(kw)
    return pace._LinattnDesc(*[a[n] for n, _ in pace._LinattnDesc._fields_])


BAD_LIN = [
    (dict(num_seqs=0), 1), (dict(num_heads=0), 1), (dict(num_heads=257), 1), (dict(io_dtype=2), 1), (dict(d_k=0, d_v=0), 1),
    (dict(d_v=32), 2), (dict(d_k=96, d_v=96), 2), (dict(d_k=256, d_v=256), 2), (dict(total_tokens=-1), 1), (dict(max_len=-1), 1),
    (dict(total_tokens=1 << 31), 2), (dict(q_stride=255), 1), (dict(k_stride=-256), 1), (dict(v_stride=1 << 31), 1),
    (dict(o_stride=1), 1), (dict(num_seqs=1 << 28, num_heads=256), 2),
]


@pytest.mark.parametrize("kw,status", BAD_LIN)
def test_linattn_descriptor(kw, status):
    d = lin(**kw)
    n = ctypes.c_size_t()
    for back in (0, 1):
        assert pace.lib.pace_linattn_workspace_bytes(ctypes.byref(d), back, ctypes.byref(n)) == status
    assert pace.lib.pace_linattn_forward(ctypes.byref(d), P, P, P, P, P, None, P, None, None, None, None) == status
    assert pace.lib.pace_linattn_backward(ctypes.byref(d), P, P, P, P, P, None, P, None, P, P, P, None, None, None,
                                          None) == status
    if "total_tokens" not in kw and "max_len" not in kw:
        assert pace.lib.pace_linattn_step(ctypes.byref(d), P, P, P, P, P, P, None) == status


def test_linattn_pointers():
    d = lin()
    good = [P] * 4 + [None, None, P, None, None, None, None]       # q k v decay cu S0 o ST ws flags stream
    for i, bad in [(0, None), (1, None), (2, None), (3, None), (6, None), (0, ODD), (6, ODD), (3, ODD), (4, ODD), (5, OFF4),
                   (7, OFF4), (8, OFF4), (9, ODD)]:
        a = list(good)
        a[i] = bad
        assert pace.lib.pace_linattn_forward(ctypes.byref(d), *a) == 1, (i, bad)
    # without cu_seqlens the rows are num_seqs * max_len
    assert pace.lib.pace_linattn_forward(ctypes.byref(lin(total_tokens=21)), *good) == 1
    assert pace.lib.pace_linattn_forward(None, *good) == 1
    good = [P] * 4 + [None, None, P, None, P, P, P, None, None, None, None]   # .. cu S0 do dST dq dk dv dS0 ws flags stream
    for i, bad in [(6, None), (8, None), (9, None), (10, None), (7, OFF4), (11, OFF4), (8, ODD)]:
        a = list(good)
        a[i] = bad
        assert pace.lib.pace_linattn_backward(ctypes.byref(d), *a) == 1, (i, bad)
    a = list(good)
    a[7] = a[11] = P                                                # dS0 over dST
    assert pace.lib.pace_linattn_backward(ctypes.byref(d), *a) == 1
    a = list(good)
    a[5] = a[11] = P                                                # dS0 over S0
    assert pace.lib.pace_linattn_backward(ctypes.byref(d), *a) == 1
    good = [P] * 6 + [None]
    for i in range(6):
        a = list(good)
        a[i] = None
        assert pace.lib.pace_linattn_step(ctypes.byref(d), *a) == 1, i
    assert pace.lib.pace_linattn_step(ctypes.byref(d), OFF4, *good[1:]) == 1


def norm(**kw):
    a = dict(num_tokens=5, num_q_heads=4, num_k_heads=2, head_dim=64, rotary_dim=0, interleaved=0, norm=1, io_dtype=0,
             eps=1e-6, q_scale=1.0, q_stride=0, k_stride=0, q_out_stride=0, k_out_stride=0)
    a.update(kw)
    return pace._QkNormDesc(*[a[n] for n, _ in pace._QkNormDesc._fields_])


@pytest.mark.parametrize("kw,status", [
    (dict(num_tokens=-1), 1), (dict(num_q_heads=-1), 1), (dict(num_q_heads=257), 1), (dict(num_q_heads=0, num_k_heads=0), 1),
    (dict(head_dim=0), 1), (dict(head_dim=60), 2), (dict(head_dim=264), 2), (dict(rotary_dim=66), 1), (dict(rotary_dim=31), 1),
    (dict(rotary_dim=-2), 1), (dict(interleaved=2), 1), (dict(norm=2), 1), (dict(io_dtype=5), 1), (dict(eps=0.0), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(q_scale=float("nan")), 1),
    (dict(q_stride=255), 1), (dict(k_stride=127), 1), (dict(q_out_stride=-1), 1), (dict(k_out_stride=(1 << 30) + 1), 1),
    (dict(num_tokens=1 << 31), 2),
])
def test_qk_norm_descriptor(kw, status):
    d = norm(**kw)
    n = ctypes.c_size_t()
    assert pace.lib.pace_qk_norm_workspace_bytes(ctypes.byref(d), ctypes.byref(n)) == status
    assert pace.lib.pace_qk_norm_rotate(ctypes.byref(d), P, P, None, None, P, P, P, P, None) == status
    assert pace.lib.pace_qk_norm_rotate_backward(ctypes.byref(d), P, P, None, None, P, P, P, P, P, P, None, None, None,
                                                 None) == status


def test_qk_norm_pointers():
    d = norm(rotary_dim=32)
    good = [P, P, None, None, P, P, P + 4096, P + 8192, None]       # q k wq wk pos inv qo ko stream
    for i, bad in [(0, None), (1, None), (4, None), (5, None), (6, None), (7, None), (0, ODD), (2, ODD), (5, ODD), (6, ODD)]:
        a = list(good)
        a[i] = bad
        assert pace.lib.pace_qk_norm_rotate(ctypes.byref(d), *a) == 1, (i, bad)
    # in place wants equal strides
    a = list(good)
    a[6] = P
    assert pace.lib.pace_qk_norm_rotate(ctypes.byref(norm(rotary_dim=32, q_out_stride=512)), *a) == 1
    good = [P, P, None, None, P, P, P, P, P + 4096, P + 8192, None, None, None, None]
    for i, bad in [(6, None), (7, None), (8, None), (10, P), (11, P), (12, ODD)]:     # a weight gradient wants workspace
        a = list(good)
        a[i] = bad
        if i == 12:
            a[10] = P
        assert pace.lib.pace_qk_norm_rotate_backward(ctypes.byref(d), *a) == 1, (i, bad)


def test_workspace_sizes():
    n = pace.pace_linattn_workspace_bytes(4, 8, 128, pace.PACE_IO_BF16, 4000, 1000, True)
    assert n % 256 == 0 and n >= 0
    assert pace.pace_qk_norm_workspace_bytes(100, 4, 2, 64, 0) % 256 == 0


def test_binding_refuses_host_tensors_and_wrong_shapes():
    q = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):
        pace.pace_linattn_forward(q, q, q, torch.zeros(2))
    with pytest.raises(ValueError):
        pace.pace_linattn_step(torch.zeros(4, 2, 64, 64), q, q, q, torch.zeros(2))
    with pytest.raises(ValueError):
        pace.pace_qk_norm_rotate(q, q)



def test_row_strides():
    """The binding's reading of a tensor's rows, on host tensors with the device check out of the way."""
    class T(torch.Tensor):
        is_cuda = True

    def rows(t, heads, d):
        t = t.as_subclass(T)
        return pace._rows("x", t, heads, d, t)

    base = torch.zeros(6, 5, 3 * 4 * 8)
    assert rows(torch.zeros(30, 4, 8), 4, 8) == (30, 32)
    assert rows(base.view(30, 12, 8)[:, 4:8], 4, 8) == (30, 96)
    assert rows(base.view(6, 5, 12, 8)[:, :, :4], 4, 8) == (30, 96)
    assert rows(torch.zeros(1, 4, 8), 4, 8) == (1, 0)
    assert rows(torch.zeros(0, 4, 8), 4, 8) == (0, 0)
    for bad in (torch.zeros(4, 8).expand(30, 4, 8),                 # one row many times
                torch.zeros(30, 8, 4).transpose(1, 2),              # heads not dense
                base.view(6, 5, 12, 8)[:, :3, :4],                  # two strides
                torch.zeros(30, 5, 8)):                             # another number of heads
        with pytest.raises(ValueError):
            rows(bad, 4, 8)


def test_binding_refuses_what_is_no_tensor_or_integer():
    q, g = torch.zeros(4, 2, 64), torch.zeros(2)
    for call in (lambda: pace.pace_linattn_forward(q.numpy(), q, q, g),
                 lambda: pace.pace_linattn_forward(q, q, q, [0.0, 0.0]),
                 lambda: pace.pace_linattn_forward(q, q, q, g, num_seqs=2.0),
                 lambda: pace.pace_linattn_backward(q, q, q, g, q, max_len="4"),
                 lambda: pace.pace_linattn_step([0], q, q, q, g),
                 lambda: pace.pace_qk_norm_rotate(q, q, rotary_dim=1.5),
                 lambda: pace.pace_qk_norm_rotate_backward(q, q, None, None, None, None, 0, q)):
        with pytest.raises(ValueError):
            call()


def test_workspace_of_the_walk_in_fp32():
    """Few heads and long sequences are cut into stretches, whose states lie in the workspace; many heads are not."""
    size = lambda n, h, d, t, back: pace.pace_linattn_workspace_bytes(n, h, d, pace.PACE_IO_F32, n * t, t, back)  # noqa: E731
    assert size(1, 1, 64, 64, False) == 0
    one = size(1, 2, 64, 4096, False)
    assert one > 0 and one % (2 * 64 * 64 * 4) == 0
    assert size(64, 32, 64, 4096, False) == size(64, 32, 64, 4096, True) == 0
    assert size(1, 1, 32, 2 ** 31 - 1, True) > 0
