"""Norms of queries and keys for each head with the position rotation (pace_qk_norm_rotate and its gradients)
against fp64, and the run of them with the linear attention."""
import numpy as np
import pytest
import torch

import bit_recurrent_state_pace_b200 as pace
from tests import operators_reference as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def make(T, hq, hk, d, rot, dt, weights, far=False, seed=1):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q, k, dq, dk = r(T, hq, d).to(dt), (3 * r(T, hk, d)).to(dt), r(T, hq, d).to(dt), r(T, hk, d).to(dt)
    wq, wk = (1 + 0.3 * r(d), 1 + 0.3 * r(d)) if weights else (None, None)
    pos = inv = None
    if rot:
        inv = torch.pow(torch.tensor(1e4, dtype=torch.float64), -2 * torch.arange(rot // 2, dtype=torch.float64) / rot).float().cuda()
        pos = (torch.randint(-(1 << 30), 1 << 30, (T,), generator=gen, device="cuda") if far else torch.arange(T, device="cuda")).int()
    return q, k, wq, wk, pos, inv, dq, dk


def tolerance(size, value, dt, d):
    """size: the largest magnitude that the channels' pair (or the row) has before the last sum.  fp32 roundings between
    input and output: d + 8 in the sum of squares (halved by the root), the root, four products, the angle's reduction to a
    half turn (2^-25 turns) and its cosine and sine (together below 8 half steps), two in the turn, and in the gradient
    as many again plus d in the inner product: below 3 d + 64 half steps."""
    t = (3 * d + 64) * ref.U32 * size
    return t if dt == torch.float32 else t + ref.UBF * (np.abs(value) + t)


def close(got, want, tol):
    got = f64(got)
    assert np.isfinite(got).all()
    over = np.abs(got - want) - tol
    assert over.max(initial=-1.0) <= 0, (float(over.max()), np.unravel_index(over.argmax(), over.shape))


def check(T, hq, hk, d, rot, inter, kind, weights, dt, far, scale, q, k, wq, wk, pos, inv, dq, dk, back=True):
    how = dict(rotary_dim=rot, interleaved=inter, norm=kind, eps=EPS, q_scale=scale)
    outs = pace.pace_qk_norm_rotate(q, k, wq, wk, pos, inv, **how)
    sides = [(q, wq, dq, scale), (k, wk, dk, 1.0)]
    for got, (x, w, _, s) in zip(outs, sides):
        want = ref.norm_rotate(f64(x), f64(w), f64(pos), f64(inv), rot, inter, kind, EPS, s)
        row = np.abs(ref.norm_rotate(f64(x), f64(w), None, None, 0, inter, kind, EPS, s)).max(-1, keepdims=True) * 2
        close(got, want, tolerance(row, want, dt, d))
    if not back:
        return
    grads = pace.pace_qk_norm_rotate_backward(q, k, wq, wk, pos, inv, dq, dk, **how)
    for got, gw, (x, w, dy, s) in zip(grads[:2], grads[2:], sides):
        want, dw, dwb = ref.norm_rotate_backward(f64(x), f64(w), f64(pos), f64(inv), rot, inter, kind, EPS, s, f64(dy))
        n = d if kind == "rms" else 1
        r = 1 / np.sqrt((f64(x) ** 2).sum(-1, keepdims=True) / n + EPS)
        wmax = 1.0 if w is None else np.abs(f64(w)).max()
        h = 2 * abs(s) * wmax * np.abs(f64(dy)).max(-1, keepdims=True)
        xh = np.abs(f64(x)) * r
        size = r * (h + xh * (xh * h).sum(-1, keepdims=True) / n)
        close(got, want, tolerance(size, want, dt, d))
        if w is None:
            assert gw is None
        else:
            # each term as above; the sum adds at most one rounding for each of its rows' terms
            rows = x.shape[0] * x.shape[1]
            urow = 2 * abs(s) * np.abs(f64(dy)).max(-1, keepdims=True) * xh
            close(gw, dw, ((3 * d + 64) * urow.sum((0, 1)) + rows * dwb) * ref.U32)


SHAPES = [(1, 1, 1, 128), (7, 4, 2, 64), (33, 5, 3, 32), (3, 32, 8, 128), (5, 2, 2, 256), (64, 1, 1, 8), (9, 3, 1, 80),
          (11, 2, 7, 24), (2, 1, 1, 96)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,hq,hk,d", SHAPES)
def test_shapes(T, hq, hk, d, inter, dt):
    for rot in sorted({0, 2, d // 4 // 2 * 2, d // 2, d}):
        for kind, weights in (("rms", True), ("l2", False)):
            far = rot == d
            check(T, hq, hk, d, rot, inter, kind, weights, DT[dt], far, 0.25, *make(T, hq, hk, d, rot, DT[dt], weights, far))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,hq,hk,d", [(3000, 16, 4, 128), (20000, 2, 1, 64), (700, 40, 40, 256), (40000, 1, 1, 32)])
def test_many_rows(T, hq, hk, d, dt):
    """More rows than one wave of blocks holds."""
    check(T, hq, hk, d, d, False, "rms", True, DT[dt], True, d ** -0.5, *make(T, hq, hk, d, d, DT[dt], True, True))


def test_far_positions_turn_as_exactly_as_near_ones():
    """The turn by 2^31 - 1 and by -2^31 positions within fp32 of the exact angle."""
    q, k, _, _, pos, inv, dq, dk = make(4, 2, 2, 64, 64, torch.float32, False)
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 0, 123456789], dtype=torch.int32, device="cuda")
    check(4, 2, 2, 64, 64, False, "l2", False, torch.float32, True, 1.0, q, k, None, None, pos, inv, dq, dk)


@pytest.mark.parametrize("off", [0, 1])
def test_parts_of_a_projection_and_in_place(off):
    T, hq, hk, d, rot, dt = 50, 4, 2, 64, 32, torch.bfloat16
    q, k, wq, wk, pos, inv, dq, dk = make(T, hq, hk, d, rot, dt, True)
    how = dict(rotary_dim=rot, norm="rms", eps=EPS, q_scale=0.5)
    want = pace.pace_qk_norm_rotate(q, k, wq, wk, pos, inv, **how)
    w = (hq + 2 * hk) * d + 8
    flat = torch.full((T * w + 8,), 7.0, dtype=dt, device="cuda")
    rows = flat[off:off + T * w].view(T, w)
    vq, vk = rows[:, :hq * d].unflatten(1, (hq, d)), rows[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
    vq.copy_(q), vk.copy_(k)
    got = pace.pace_qk_norm_rotate(vq, vk, wq, wk, pos, inv, **how)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    g0 = pace.pace_qk_norm_rotate_backward(q, k, wq, wk, pos, inv, dq, dk, **how)
    g1 = pace.pace_qk_norm_rotate_backward(vq, vk, wq, wk, pos, inv, dq, dk, **how)
    assert all(torch.equal(a, b) for a, b in zip(g0, g1))
    pace.pace_qk_norm_rotate(vq, vk, wq, wk, pos, inv, q_out=vq, k_out=vk, **how)
    assert torch.equal(vq, want[0]) and torch.equal(vk, want[1]) and bool((rows[:, (hq + hk) * d:] == 7.0).all())
    a, b = dq.clone(), dk.clone()
    g2 = pace.pace_qk_norm_rotate_backward(q, k, wq, wk, pos, inv, a, b, dq=a, dk=b, **how)
    assert all(torch.equal(x, y) for x, y in zip(g0, g2))


def test_one_side_only_and_no_tokens():
    q, k, wq, wk, pos, inv, dq, dk = make(6, 3, 2, 64, 64, torch.bfloat16, True)
    how = dict(rotary_dim=64, norm="rms", eps=EPS)
    both = pace.pace_qk_norm_rotate(q, k, wq, wk, pos, inv, **how)
    assert torch.equal(pace.pace_qk_norm_rotate(q, None, wq, None, pos, inv, **how)[0], both[0])
    assert torch.equal(pace.pace_qk_norm_rotate(None, k, None, wk, pos, inv, **how)[1], both[1])
    g = pace.pace_qk_norm_rotate_backward(q, k, wq, wk, pos, inv, dq, dk, **how)
    g1 = pace.pace_qk_norm_rotate_backward(None, k, None, wk, pos, inv, None, dk, **how)
    assert g1[0] is None and g1[2] is None and torch.equal(g1[1], g[1])
    e = [x[:0] for x in (q, k, dq, dk)]
    out = pace.pace_qk_norm_rotate(e[0], e[1], wq, wk, pos[:0], inv, **how)
    assert out[0].shape == (0, 3, 64)
    g = pace.pace_qk_norm_rotate_backward(e[0], e[1], wq, wk, pos[:0], inv, e[2], e[3], **how)
    assert bool((g[2] == 0).all()) and bool((g[3] == 0).all())


def test_zero_rows_and_nan_rows_stay_to_themselves():
    q, k, wq, wk, pos, inv, dq, dk = make(8, 4, 2, 128, 64, torch.bfloat16, True)
    how = dict(rotary_dim=64, norm="l2", eps=EPS)
    want = pace.pace_qk_norm_rotate(q, k, wq, wk, pos, inv, **how)
    q[2, 1] = 0
    q[5, 3] = float("nan")
    k[1, 0, 7] = float("inf")
    got = pace.pace_qk_norm_rotate(q, k, wq, wk, pos, inv, **how)
    assert bool((got[0][2, 1] == 0).all()) and bool(torch.isnan(got[0][5, 3]).all()) and bool(torch.isnan(got[1][1, 0]).any())
    keep = torch.ones(8, 4, dtype=torch.bool, device="cuda")
    keep[2, 1] = keep[5, 3] = False
    assert torch.equal(got[0][keep], want[0][keep])
    keep = torch.ones(8, 2, dtype=torch.bool, device="cuda")
    keep[1, 0] = False
    assert torch.equal(got[1][keep], want[1][keep])


def test_gradient_by_differences():
    """Central differences of the fp64 form with step 1e-4: truncation below 1e-7 of the sums here, fp64 rounding below
    1e-10, against the kernel's fp32 gradients."""
    T, hq, hk, d, rot = 5, 2, 1, 32, 16
    q, k, wq, wk, pos, inv, dq, dk = make(T, hq, hk, d, rot, torch.float32, True)
    how = dict(rotary_dim=rot, interleaved=True, norm="rms", eps=EPS, q_scale=0.5)
    gx, _, gw, _ = pace.pace_qk_norm_rotate_backward(q, k, wq, wk, pos, inv, dq, dk, **how)
    rng = np.random.default_rng(3)
    ex, ew = rng.standard_normal(q.shape), rng.standard_normal(d)

    def loss(x, w):
        return float((ref.norm_rotate(x, w, f64(pos), f64(inv), rot, True, "rms", EPS, 0.5) * f64(dq)).sum())

    h = 1e-4
    nx = (loss(f64(q) + h * ex, f64(wq)) - loss(f64(q) - h * ex, f64(wq))) / (2 * h)
    nw = (loss(f64(q), f64(wq) + h * ew) - loss(f64(q), f64(wq) - h * ew)) / (2 * h)
    size = float((np.abs(f64(gx)) * np.abs(ex)).sum())
    assert abs(float((f64(gx) * ex).sum()) - nx) <= ((3 * d + 64) * ref.U32 * 8 + 1e-7) * size
    size = float((np.abs(f64(gw)) * np.abs(ew)).sum())
    assert abs(float((f64(gw) * ew).sum()) - nw) <= ((3 * d + 64) * ref.U32 * 8 + 1e-7) * size


def test_same_bits_graph_and_streams():
    T, hq, hk, d, rot, dt = 400, 8, 4, 128, 128, torch.bfloat16
    args, args2 = make(T, hq, hk, d, rot, dt, True), make(T, hq, hk, d, rot, dt, True, seed=2)
    how = dict(rotary_dim=rot, norm="rms", eps=EPS)

    def all_of(a, stream=None):
        return (pace.pace_qk_norm_rotate(*a[:6], stream=stream, **how)
                + pace.pace_qk_norm_rotate_backward(*a, stream=stream, **how))

    want, want2 = all_of(args), all_of(args2)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    got, got2 = all_of(args, sa), all_of(args2, sb)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want + want2, got + got2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = all_of(args)
    for x, y in zip(args, args2):
        x.copy_(y)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want2, held))


def test_refusals():
    q, k, wq, wk, pos, inv, dq, dk = make(6, 3, 2, 64, 64, torch.bfloat16, True)
    how = dict(rotary_dim=64)
    for call in (lambda: pace.pace_qk_norm_rotate(q, k[:5], wq, wk, pos, inv, **how),
                 lambda: pace.pace_qk_norm_rotate(q, k.float(), wq, wk, pos, inv, **how),
                 lambda: pace.pace_qk_norm_rotate(q, k, wq[:8], wk, pos, inv, **how),
                 lambda: pace.pace_qk_norm_rotate(q, k, wq, wk, pos.long(), inv, **how),
                 lambda: pace.pace_qk_norm_rotate(q, k, wq, wk, pos[:4], inv, **how),
                 lambda: pace.pace_qk_norm_rotate(q, k, wq, wk, pos, inv[:4], **how),
                 lambda: pace.pace_qk_norm_rotate(q, k, wq, wk, None, inv, **how),
                 lambda: pace.pace_qk_norm_rotate(q, k, wq, wk, pos, inv, norm="max", **how),
                 lambda: pace.pace_qk_norm_rotate_backward(q, k, wq, wk, pos, inv, dq, None, **how)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(pace.PaceError) as e:
        pace.pace_qk_norm_rotate(q, k, eps=0.0)
    assert e.value.status == pace.PACE_ERR_INVALID_ARG


def test_together_as_a_layer_uses_them():
    """Projection rows -> normalised and turned q, k -> prompts -> single tokens, and the way back to the projection's
    gradient, in fp32 against fp64 with the library's own intermediate values as inputs of each step."""
    N, T, H, d, rot = 2, 90, 3, 64, 32
    gen = torch.Generator(device="cuda").manual_seed(9)
    proj = torch.randn(N * T, 3, H, d, generator=gen, device="cuda")
    rows = proj.view(N * T, -1)
    q, k, v = (x.unflatten(1, (H, d)) for x in rows.split(H * d, 1))
    wq, wk = 1 + 0.1 * torch.randn(d, generator=gen, device="cuda"), 1 + 0.1 * torch.randn(d, generator=gen, device="cuda")
    inv = torch.pow(torch.tensor(1e4), -2 * torch.arange(rot // 2) / rot).float().cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda").repeat(N)
    g = torch.tensor([-0.5, -0.05, -0.005], device="cuda")
    how = dict(rotary_dim=rot, norm="rms", eps=EPS, q_scale=d ** -0.5)
    qn, kn = pace.pace_qk_norm_rotate(q, k, wq, wk, pos, inv, **how)
    o, ST = pace.pace_linattn_forward(qn, kn, v, g, num_seqs=N)
    do, dST = torch.randn(N * T, H, d, generator=gen, device="cuda"), torch.randn(N, H, d, d, generator=gen, device="cuda")
    grad = torch.zeros_like(rows)
    gq, gk, gv = (x.unflatten(1, (H, d)) for x in grad.split(H * d, 1))
    dqn, dkn, dv, _ = pace.pace_linattn_backward(qn, kn, v, g, do, dv=gv, num_seqs=N, dST=dST)
    _, _, dwq, dwk = pace.pace_qk_norm_rotate_backward(q, k, wq, wk, pos, inv, dqn, dkn, dq=gq, dk=gk, **how)
    # the whole of it in fp64
    p64 = proj.double().cpu().requires_grad_()
    w64 = [w.double().cpu().requires_grad_() for w in (wq, wk)]
    ang = pos.double().cpu()[:, None, None] * inv.double().cpu()

    def one(x, w, s):
        y = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        return s * torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin(), y[..., rot:]], -1)

    q6, k6, v6 = one(p64[:, 0], w64[0], d ** -0.5), one(p64[:, 1], w64[1], 1.0), p64[:, 2]
    a = g.double().cpu().exp()[None, :, None, None]
    S, outs = torch.zeros(N, H, d, d, dtype=torch.float64), []
    q6, k6, v6 = (x.view(N, T, H, d) for x in (q6, k6, v6))
    for t in range(T):
        S = a * S + v6[:, t, :, :, None] * k6[:, t, :, None, :]
        outs.append((S * q6[:, t, :, None, :]).sum(-1))
    o6 = torch.stack(outs, 1).view(N * T, H, d)
    ((o6 * do.double().cpu()).sum() + (S * dST.double().cpu()).sum()).backward()

    def off(x, y):
        return float((x.double().cpu() - y.detach()).norm() / y.detach().norm())

    # two operators after one another: the roundings of both, each below roundings32 half steps of sums whose terms
    # exceed them at most sqrt(T d)-fold here; in the norm over all values they average out to far less than
    tol = 2 * ref.roundings32(T, d) * ref.U32
    assert off(o, o6) <= tol and off(ST, S) <= tol
    assert off(grad.view_as(proj), p64.grad) <= tol
    assert off(dwq, w64[0].grad) <= tol and off(dwk, w64[1].grad) <= tol
    # and on, token by token
    x = torch.randn(N, 3, H, d, generator=gen, device="cuda")
    at = torch.full((N,), T, dtype=torch.int32, device="cuda")
    qt, kt = pace.pace_qk_norm_rotate(x[:, 0], x[:, 1], wq, wk, at, inv, **how)
    S_before = ST.clone()
    ot = pace.pace_linattn_step(ST, qt, kt, x[:, 2], g)
    S_want = a * S_before.double().cpu() + x[:, 2].double().cpu()[..., :, None] * kt.double().cpu()[..., None, :]
    assert off(ST, S_want) <= tol and off(ot, (S_want * qt.double().cpu()[..., None, :]).sum(-1)) <= tol


def test_numbers_given_as_tensors_are_read_on_every_call():
    q = make(5, 2, 2, 64, 0, torch.float32, False)[0]
    scale = torch.tensor(2.0)
    twice, _ = pace.pace_qk_norm_rotate(q, None, q_scale=scale)
    scale.fill_(3.0)
    thrice, _ = pace.pace_qk_norm_rotate(q, None, q_scale=scale)
    plain = pace.pace_qk_norm_rotate(q, None)[0]
    # a product of a unit by 2 is exact; by 3 it is rounded where the kernel rounds it
    assert torch.equal(twice, 2 * plain)
    assert bool((thrice - 3 * plain).abs().le(4 * ref.U32 * 3 * plain.abs()).all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_offsets_beyond_32_bits(dt):
    """Rows so far apart that the last ones lie more than 2^31 elements behind the first: what packed rows give."""
    dt, T, d, far = DT[dt], 140, 64, 1 << 24
    q, k, wq, wk, pos, inv, dq, dk = make(T, 1, 2, d, d, dt, True)
    how = dict(rotary_dim=d, norm="rms", eps=EPS)
    want = pace.pace_qk_norm_rotate(q, k, wq, wk, pos, inv, **how)
    want_g = pace.pace_qk_norm_rotate_backward(q, k, wq, wk, pos, inv, dq, dk, **how)
    room = torch.empty(T * far, device="cuda", dtype=dt).view(T, far)
    parts, at = [], 0
    for heads in (1, 2, 1, 2):
        parts.append(room[:, at * d:(at + heads) * d].unflatten(1, (heads, d)))
        at += heads
    parts[0].copy_(q)
    parts[1].copy_(k)
    got = pace.pace_qk_norm_rotate(parts[0], parts[1], wq, wk, pos, inv, q_out=parts[2], k_out=parts[3], **how)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = pace.pace_qk_norm_rotate_backward(parts[0], parts[1], wq, wk, pos, inv, dq, dk, dq=parts[2], dk=parts[3], **how)
    assert all(torch.equal(a, b) for a, b in zip(got, want_g))
