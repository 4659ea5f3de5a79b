"""Linear attention with a fixed decay for each head (pace_linattn_forward / _backward / _step) against fp64."""
import numpy as np
import pytest
import torch

import bit_recurrent_state_pace_b200 as pace
from tests import operators_reference as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def decays(H, seed=0):
    """From no memory at all to no forgetting."""
    g = -torch.exp2(-8.0 * torch.arange(1, H + 1, dtype=torch.float64) / H).float()
    if H >= 3:
        g[0], g[1] = float("-inf"), 0.0
    return g.cuda()


def make(total, H, d, dt, n, seed=1, states=True):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    u = lambda x: x / x.square().sum(-1, keepdim=True).sqrt()  # noqa: E731
    q, k, v, do = u(r(total, H, d)).to(dt), u(r(total, H, d)).to(dt), r(total, H, d).to(dt), r(total, H, d).to(dt)
    S0, dST = (r(n, H, d, d), r(n, H, d, d)) if states else (None, None)
    return q, k, v, do, S0, dST


def zeros(n, H, d):
    return np.zeros((n, H, d, d))


def io_tol(bound, value, dt, longest, d):
    """fp32: one rounding each (operators_reference).  bf16: the score or the state is rounded to bf16 as an operand of
    the second product (once for each term, so 2^-8 of the bound) and the output once; the rest is fp32."""
    t = ref.roundings32(longest, d) * ref.U32 * bound
    return t if dt == torch.float32 else t + ref.UBF * bound + ref.UBF * (np.abs(value) + ref.UBF * bound)


def state_tol(bound, longest, d):
    """States are sums of 32-bit products in either type (the bf16 operands are split so that 24 bits are kept)."""
    return ref.roundings32(longest, d) * ref.U32 * bound


# The tolerances count relative half steps, which subnormal numbers do not keep to: there a rounding is off by half a
# step of 2^-149 (fp32) or 2^-133 (a bf16 part), whatever the number.  At most roundings32(5000, 128) < 2^15 of them, each
# times a further factor below 2^3 (inputs of these tests), add up to less than 2^(15 - 134 + 3).
TINY = 2.0 ** -116


def close(got, want, tol):
    got = f64(got)
    assert np.isfinite(got).all()
    over = np.abs(got - want) - tol - TINY
    assert over.max(initial=-1.0) <= 0, (float(over.max()), np.unravel_index(over.argmax(), over.shape))


def check_forward(q, k, v, g, S0, cu, o, ST, dt):
    n, H, d = len(cu) - 1, q.shape[-2], q.shape[-1]
    longest = max([e - b for b, e in zip(cu[:-1], cu[1:])] + [1])
    s0 = f64(S0) if S0 is not None else zeros(n, H, d)
    wo, ws, bo, bs = ref.forward(f64(q), f64(k), f64(v), f64(g), s0, cu)
    rows = np.zeros(q.shape[0], dtype=bool)
    for b, e in zip(cu[:-1], cu[1:]):
        rows[b:e] = True
    close(o[torch.from_numpy(rows).cuda()], wo[rows], io_tol(bo, wo, dt, longest, d)[rows])
    if ST is not None:
        close(ST, ws, state_tol(bs, longest, d))


def check_backward(q, k, v, g, S0, do, dST, cu, grads, dt):
    n, H, d = len(cu) - 1, q.shape[-2], q.shape[-1]
    longest = max([e - b for b, e in zip(cu[:-1], cu[1:])] + [1])
    s0 = f64(S0) if S0 is not None else zeros(n, H, d)
    dst = f64(dST) if dST is not None else zeros(n, H, d)
    want = ref.backward(f64(q), f64(k), f64(v), f64(g), s0, f64(do), dst, cu)
    rows = np.zeros(q.shape[0], dtype=bool)
    for b, e in zip(cu[:-1], cu[1:]):
        rows[b:e] = True
    pick = torch.from_numpy(rows).cuda()
    for got, (w, b) in zip(grads[:3], want[:3]):
        close(got[pick], w[rows], io_tol(b, w, dt, longest, d)[rows])
    if grads[3] is not None:
        close(grads[3], want[3][0], state_tol(want[3][1], longest, d))


LENGTHS = [[1], [2, 1], [63], [64], [65], [0, 5, 0], [128, 127, 129, 0, 1, 64], [200], [0]]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("lens", LENGTHS, ids=str)
def test_ragged(lens, d, dt):
    """Lengths of zero and one, ends inside and at chunk edges, with states in and out, forwards and backwards."""
    dt, H, n = DT[dt], 3, len(lens)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    q, k, v, do, S0, dST = make(int(cu[-1]), H, d, dt, n)
    g, dev_cu = decays(H), torch.from_numpy(cu.astype(np.int32)).cuda()
    o, ST = pace.pace_linattn_forward(q, k, v, g, cu_seqlens=dev_cu, max_len=max(lens), S0=S0)
    check_forward(q, k, v, g, S0, cu, o, ST, dt)
    grads = pace.pace_linattn_backward(q, k, v, g, do, cu_seqlens=dev_cu, max_len=max(lens), S0=S0, dST=dST)
    check_backward(q, k, v, g, S0, do, dST, cu, grads, dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("d,n,T,H", [(128, 1, 700, 2), (64, 2, 513, 1), (32, 3, 100, 5), (128, 5, 96, 40)])
def test_uniform_without_states(d, n, T, H, dt):
    """Prompts of one length, empty states before them; [N, T, H, d] and packed rows give the same."""
    dt = DT[dt]
    cu = np.arange(n + 1) * T
    q, k, v, do, _, _ = make(n * T, H, d, dt, n, states=False)
    g = decays(H)
    o, ST = pace.pace_linattn_forward(q, k, v, g, num_seqs=n)
    check_forward(q, k, v, g, None, cu, o, ST, dt)
    o4, ST4 = pace.pace_linattn_forward(*(x.view(n, T, H, d) for x in (q, k, v)), g)
    assert torch.equal(o4.view_as(o), o) and torch.equal(ST4, ST)
    grads = pace.pace_linattn_backward(q, k, v, g, do, num_seqs=n)
    assert grads[3] is None
    check_backward(q, k, v, g, None, do, None, cu, grads, dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_long(d, dt):
    """One long sequence of few heads, which the library may cut into stretches: continues from S0 into ST, and its
    gradients, against the recurrence."""
    dt, H, T = DT[dt], 2, 5000
    q, k, v, do, S0, dST = make(T, H, d, dt, 1, seed=3)
    g, cu = torch.tensor([-0.3, -0.002], device="cuda"), np.array([0, T])
    o, ST = pace.pace_linattn_forward(q, k, v, g, S0=S0)
    check_forward(q, k, v, g, S0, cu, o, ST, dt)
    grads = pace.pace_linattn_backward(q, k, v, g, do, S0=S0, dST=dST)
    check_backward(q, k, v, g, S0, do, dST, cu, grads, dt)


def test_max_len_only_guides():
    """Results hold for sequences longer than max_len says."""
    cu = np.array([0, 700, 1500])
    q, k, v, do, S0, dST = make(1500, 2, 128, torch.bfloat16, 2)
    g, dev_cu = decays(2), torch.from_numpy(cu.astype(np.int32)).cuda()
    for most in (0, 1, 64, 5000):
        o, ST = pace.pace_linattn_forward(q, k, v, g, cu_seqlens=dev_cu, max_len=most, S0=S0)
        check_forward(q, k, v, g, S0, cu, o, ST, torch.bfloat16)
        grads = pace.pace_linattn_backward(q, k, v, g, do, cu_seqlens=dev_cu, max_len=most, S0=S0, dST=dST)
        check_backward(q, k, v, g, S0, do, dST, cu, grads, torch.bfloat16)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("off", [0, 1])
def test_parts_of_a_projection(off, dt):
    """q, k and v as parts of one projection's rows (off = 1: at addresses of element alignment only), o and the
    gradients into parts of wider rows, whose other elements stay."""
    dt, H, d, T = DT[dt], 2, 64, 150
    cu = np.array([0, 90, T])
    q, k, v, do, S0, dST = make(T, H, d, dt, 2)
    g, dev_cu, w = decays(H), torch.from_numpy(cu.astype(np.int32)).cuda(), H * d

    def wide(parts):
        flat = torch.full((T * (len(parts) * w + 8) + 8,), 7.0, device="cuda", dtype=dt)
        rows = flat[off:off + T * (len(parts) * w + 8)].view(T, -1)
        views = [rows[:, i * w:(i + 1) * w].unflatten(1, (H, d)) for i in range(len(parts))]
        for x, y in zip(views, parts):
            x.copy_(y)
        return flat, rows, views

    _, _, (wq, wk, wv) = wide([q, k, v])
    flat_o, rows_o, (wo, wdo) = wide([torch.zeros_like(q), do])
    before = rows_o[:, w:].clone()
    o, ST = pace.pace_linattn_forward(wq, wk, wv, g, o=wo, cu_seqlens=dev_cu, max_len=90, S0=S0)
    assert o is wo
    check_forward(q, k, v, g, S0, cu, wo, ST, dt)
    assert torch.equal(rows_o[:, w:], before)
    flat_g, rows_g, (dq, dk, dv) = wide([torch.zeros_like(q)] * 3)
    grads = pace.pace_linattn_backward(wq, wk, wv, g, wdo, dq=dq, dk=dk, dv=dv, cu_seqlens=dev_cu, max_len=90, S0=S0,
                                       dST=dST)
    check_backward(q, k, v, g, S0, do, dST, cu, grads, dt)
    assert bool((rows_g[:, 3 * w:] == 7.0).all())
    made = pace.pace_linattn_backward(wq, wk, wv, g, wdo, cu_seqlens=dev_cu, max_len=90, S0=S0, dST=dST)
    assert all(torch.equal(a, b) for a, b in zip(made, grads))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_rows_of_no_sequence_stay(dt):
    """Rows before the first, between and behind the sequences: not read (they hold NaN), not written."""
    dt, H, d = DT[dt], 2, 128
    cu = [5, 70, 70, 140]
    T = 200
    q, k, v, do, S0, dST = make(T, H, d, dt, 3)
    for x in (q, k, v, do):
        x[:5] = float("nan")
        x[140:] = float("nan")
    g, dev_cu = decays(H), torch.tensor(cu, dtype=torch.int32, device="cuda")
    o = torch.full_like(q, 7.0)
    _, ST = pace.pace_linattn_forward(q, k, v, g, o=o, cu_seqlens=dev_cu, max_len=70, S0=S0)
    clean = [torch.nan_to_num(x, nan=0.0) for x in (q, k, v, do)]
    check_forward(*clean[:3], g, S0, cu, o, ST, dt)
    out = [torch.full_like(q, 7.0) for _ in range(3)]
    grads = pace.pace_linattn_backward(q, k, v, g, do, dq=out[0], dk=out[1], dv=out[2], cu_seqlens=dev_cu, max_len=70,
                                       S0=S0, dST=dST)
    check_backward(*clean[:3], g, S0, clean[3], dST, cu, grads, dt)
    for x in (o, *out):
        assert bool((x[:5] == 7.0).all()) and bool((x[140:] == 7.0).all())


def test_neighbours_do_not_mix():
    """A NaN of one sequence, and of one head, stays there."""
    cu = [0, 70, 150, 200]
    q, k, v, do, S0, dST = make(200, 3, 128, torch.bfloat16, 3)
    g, dev_cu = decays(3), torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, ST = pace.pace_linattn_forward(q, k, v, g, cu_seqlens=dev_cu, max_len=80, S0=S0)
    for t in (71, 149):                                         # second sequence, head 1
        for x in (q, k, v):
            x[t, 1] = float("nan")
    o2, ST2 = pace.pace_linattn_forward(q, k, v, g, cu_seqlens=dev_cu, max_len=80, S0=S0)
    keep = torch.ones(200, 3, dtype=torch.bool, device="cuda")
    keep[70:150, 1] = False
    assert torch.equal(o[keep], o2[keep])
    assert torch.equal(ST[[0, 2]], ST2[[0, 2]]) and torch.equal(ST[1][[0, 2]], ST2[1][[0, 2]])
    assert bool(torch.isnan(ST2[1, 1]).any()) and bool(torch.isnan(o2[149, 1]).all())


def test_offsets_out_of_range_are_held():
    """Offsets outside the rows are moved to their edge, a sequence that ends before it begins is empty."""
    q, k, v, do, S0, dST = make(100, 2, 128, torch.bfloat16, 3)
    g = decays(2)
    wild = torch.tensor([-50, 40, 30, 1 << 30], dtype=torch.int32, device="cuda")
    o, ST = pace.pace_linattn_forward(q, k, v, g, cu_seqlens=wild, max_len=100, S0=S0)
    _, ST1 = pace.pace_linattn_forward(q[:40], k[:40], v[:40], g, S0=S0[:1])
    assert torch.equal(ST[:1], ST1) and torch.equal(ST[1], S0[1])
    o3, ST3 = pace.pace_linattn_forward(q[30:], k[30:], v[30:], g, S0=S0[2:])
    assert torch.equal(ST[2:], ST3) and torch.equal(o[40:], o3[10:])


def test_state_in_place_and_none():
    """ST over S0; ST not wanted; prompts continued in two calls give what one call gives."""
    q, k, v, do, S0, _ = make(300, 2, 128, torch.bfloat16, 1)
    g = decays(2)
    o, ST = pace.pace_linattn_forward(q, k, v, g, S0=S0)
    S = S0.clone()
    o2, same = pace.pace_linattn_forward(q, k, v, g, S0=S, ST=S)
    assert same is S and torch.equal(S, ST) and torch.equal(o, o2)
    o3, none = pace.pace_linattn_forward(q, k, v, g, S0=S0, need_ST=False)
    assert none is None and torch.equal(o, o3)
    S = S0.clone()
    parts = [pace.pace_linattn_forward(q[b:e], k[b:e], v[b:e], g, S0=S, ST=S)[0] for b, e in ((0, 101), (101, 300))]
    check_forward(q, k, v, g, S0, [0, 300], torch.cat(parts), S, torch.bfloat16)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("n,H", [(1, 1), (3, 5), (2, 32), (70, 7)])
def test_step(n, H, d, dt):
    dt = DT[dt]
    q, k, v, _, S0, _ = make(n, H, d, dt, n)
    g = decays(H)
    S = S0.clone()
    o = pace.pace_linattn_step(S, q, k, v, g)
    cu = np.arange(n + 1)
    wo, ws, bo, bs = ref.forward(f64(q), f64(k), f64(v), f64(g), f64(S0), cu)
    close(S, ws, ref.roundings32(1, d) * ref.U32 * bs)
    tol = ref.roundings32(1, d) * ref.U32 * bo
    if dt == torch.bfloat16:
        tol = tol + ref.UBF * (np.abs(wo) + tol)
    close(o, wo, tol)


def test_step_from_parts_of_a_projection():
    n, H, d = 9, 4, 64
    q, k, v, _, S0, _ = make(n, H, d, torch.bfloat16, n)
    rows = torch.cat([x.reshape(n, -1) for x in (q, k, v)], 1)
    views = [x.unflatten(1, (H, d)) for x in rows.split(H * d, 1)]
    g, Sa, Sb = decays(H), S0.clone(), S0.clone()
    assert torch.equal(pace.pace_linattn_step(Sa, q, k, v, g), pace.pace_linattn_step(Sb, *views, g))
    assert torch.equal(Sa, Sb)


def test_prompt_then_tokens():
    """A prompt's state goes on token by token as the prompt continued would."""
    T, more, H, d = 130, 6, 3, 128
    q, k, v, _, S0, _ = make(2 * (T + more), H, d, torch.float32, 2)
    q4, k4, v4 = (x.view(2, T + more, H, d) for x in (q, k, v))
    g = decays(H)
    o, ST = pace.pace_linattn_forward(*(x[:, :T].contiguous() for x in (q4, k4, v4)), g, S0=S0)
    outs = [o] + [pace.pace_linattn_step(ST, *(x[:, t].contiguous() for x in (q4, k4, v4)), g)[:, None]
                  for t in range(T, T + more)]
    cu = np.arange(3) * (T + more)
    check_forward(q, k, v, g, S0, cu, torch.cat(outs, 1).reshape(-1, H, d), ST, torch.float32)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_gradient_by_differences(dt):
    """Directional derivatives of a loss of o and ST, by central differences of the fp64 recurrence, against the
    kernels' gradients.  The loss is linear in each input alone, so the differences carry no truncation error; what is
    left is the gradients' own tolerance."""
    dt, T, H, d = DT[dt], 75, 2, 64
    q, k, v, do, S0, dST = make(T, H, d, dt, 1, seed=11)
    g, cu = torch.tensor([-0.1, -0.01], device="cuda"), [0, T]
    dq, dk, dv, dS0 = pace.pace_linattn_backward(q, k, v, g, do, S0=S0, dST=dST)
    x = dict(q=f64(q), k=f64(k), v=f64(v), S0=f64(S0))
    want = ref.backward(x["q"], x["k"], x["v"], f64(g), x["S0"], f64(do), f64(dST), cu)

    def loss(**over):
        y = dict(x, **over)
        o, ST, _, _ = ref.forward(y["q"], y["k"], y["v"], f64(g), y["S0"], cu)
        return float((o * f64(do)).sum() + (ST * f64(dST)).sum())

    rng = np.random.default_rng(5)
    for (name, got), (w, b) in zip((("q", dq), ("k", dk), ("v", dv), ("S0", dS0)), want):
        e = rng.standard_normal(x[name].shape)
        numeric = (loss(**{name: x[name] + e}) - loss(**{name: x[name] - e})) / 2
        tol = state_tol(b, T, d) if name == "S0" else io_tol(b, w, dt, T, d)
        assert abs(float((f64(got) * e).sum()) - numeric) <= float((np.abs(e) * tol).sum()) + 1e-9 * abs(numeric), name


def test_same_bits_twice():
    q, k, v, do, S0, dST = make(900, 3, 128, torch.bfloat16, 1)
    g = decays(3)
    a = pace.pace_linattn_forward(q, k, v, g, S0=S0) + pace.pace_linattn_backward(q, k, v, g, do, S0=S0, dST=dST)
    b = pace.pace_linattn_forward(q, k, v, g, S0=S0) + pace.pace_linattn_backward(q, k, v, g, do, S0=S0, dST=dST)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("T,H", [(300, 3), (4000, 1)])
def test_graph_and_streams(T, H):
    """Captured and replayed on new inputs; on a stream of its own; two streams at once with a workspace each."""
    d, dt = 128, torch.bfloat16
    q, k, v, do, S0, dST = make(T, H, d, dt, 1)
    q2, k2, v2, do2, S02, dST2 = make(T, H, d, dt, 1, seed=2)
    g = decays(H)

    def all_of(q, k, v, do, S0, dST, stream=None):
        return (pace.pace_linattn_forward(q, k, v, g, S0=S0, stream=stream)
                + pace.pace_linattn_backward(q, k, v, g, do, S0=S0, dST=dST, stream=stream))

    want, want2 = all_of(q, k, v, do, S0, dST), all_of(q2, k2, v2, do2, S02, dST2)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    got, got2 = all_of(q, k, v, do, S0, dST, sa), all_of(q2, k2, v2, do2, S02, dST2, sb.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want + want2, got + got2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = all_of(q, k, v, do, S0, dST)
        S = S0.clone()
        tok = pace.pace_linattn_step(S, q[:1], k[:1], v[:1], g)
    for x, y in zip((q, k, v, do, S0, dST), (q2, k2, v2, do2, S02, dST2)):
        x.copy_(y)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want2, held))
    S = S02.clone()
    assert torch.equal(pace.pace_linattn_step(S, q2[:1], k2[:1], v2[:1], g), tok)


def test_flags_stay_clear_and_bad_tensors_are_refused():
    q, k, v, do, S0, dST = make(64, 2, 64, torch.bfloat16, 1)
    g = decays(2)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    pace.pace_linattn_forward(q, k, v, g, S0=S0, flags=flags)
    pace.pace_linattn_backward(q, k, v, g, do, S0=S0, dST=dST, flags=flags)
    assert int(flags) == 0
    for call in (lambda: pace.pace_linattn_forward(q, k.float(), v, g),
                 lambda: pace.pace_linattn_forward(q, k[:10], v, g),
                 lambda: pace.pace_linattn_forward(q, k, v, g.double()),
                 lambda: pace.pace_linattn_forward(q, k, v, g[:1]),
                 lambda: pace.pace_linattn_forward(q, k, v, g, S0=S0[:, :1]),
                 lambda: pace.pace_linattn_forward(q, k, v, g, S0=S0.cpu()),
                 lambda: pace.pace_linattn_forward(q, k, v, g, num_seqs=3),
                 lambda: pace.pace_linattn_forward(q, k, v, g, cu_seqlens=torch.tensor([0, 64], device="cuda")),
                 lambda: pace.pace_linattn_forward(q[:, :, ::2], k, v, g),
                 lambda: pace.pace_linattn_backward(q, k, v, g, do[:3]),
                 lambda: pace.pace_linattn_step(S0, q, k, v, g)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_stretches_of_ragged_sequences(d, dt):
    """Few heads and one long sequence beside short and empty ones: some are cut into stretches, their ends inside, at and
    one behind a chunk; ST over S0."""
    dt, H, lens = DT[dt], 2, [1100, 0, 1, 64, 513, 640, 65]
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    q, k, v, do, S0, dST = make(int(cu[-1]), H, d, dt, len(lens), seed=7)
    g, dev_cu = torch.tensor([-0.05, -0.0007], device="cuda"), torch.from_numpy(cu.astype(np.int32)).cuda()
    assert pace.pace_linattn_workspace_bytes(len(lens), H, d, pace.PACE_IO_F32 if dt == torch.float32 else pace.PACE_IO_BF16,
                                             int(cu[-1]), 1100, False) > 0
    ST = S0.clone()
    o, _ = pace.pace_linattn_forward(q, k, v, g, cu_seqlens=dev_cu, max_len=1100, S0=ST, ST=ST)
    check_forward(q, k, v, g, S0, cu, o, ST, dt)
    grads = pace.pace_linattn_backward(q, k, v, g, do, cu_seqlens=dev_cu, max_len=1100, S0=S0, dST=dST)
    check_backward(q, k, v, g, S0, do, dST, cu, grads, dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n", [512, 513, 700])
def test_many_sequences(n, dt):
    """More short sequences than blocks, around the number up to which they are sorted, with states in and out."""
    dt, H, d = DT[dt], 2, 64
    lens = np.random.default_rng(n).integers(0, 100, n)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    q, k, v, do, S0, dST = make(int(cu[-1]), H, d, dt, n, seed=n)
    g, dev_cu = torch.tensor([-0.2, -0.01], device="cuda"), torch.from_numpy(cu.astype(np.int32)).cuda()
    o, ST = pace.pace_linattn_forward(q, k, v, g, cu_seqlens=dev_cu, max_len=100, S0=S0)
    check_forward(q, k, v, g, S0, cu, o, ST, dt)
    grads = pace.pace_linattn_backward(q, k, v, g, do, cu_seqlens=dev_cu, max_len=100, S0=S0, dST=dST)
    check_backward(q, k, v, g, S0, do, dST, cu, grads, dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_decays_of_every_size(d, dt):
    """Decays whose powers leave the range of fp32 within a chunk, within a few tokens, and ones that round to 1."""
    dt, T = DT[dt], 210
    g = torch.tensor([-1.3, -2.999, -3.001, -45.0, -88.0, -104.0, -1e30, -1e-8], device="cuda")
    H, cu = g.numel(), np.array([0, 150, T])
    q, k, v, do, S0, dST = make(T, H, d, dt, 2, seed=4)
    dev_cu = torch.from_numpy(cu.astype(np.int32)).cuda()
    o, ST = pace.pace_linattn_forward(q, k, v, g, cu_seqlens=dev_cu, max_len=150, S0=S0)
    check_forward(q, k, v, g, S0, cu, o, ST, dt)
    for s, t in ((S0, dST), (None, None)):
        grads = pace.pace_linattn_backward(q, k, v, g, do, cu_seqlens=dev_cu, max_len=150, S0=s, dST=t)
        check_backward(q, k, v, g, s, do, t, cu, grads, dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("d", [32, 64])
def test_large_values(d, dt):
    """Values of 1e30: nothing on the way to finite results overflows, whichever way a head's decay is applied."""
    dt, T = DT[dt], 70
    g, cu = torch.tensor([-2.9, -1.001, -0.999, -0.3, -1e-4], device="cuda"), np.array([0, T])
    q, k, v, do, S0, dST = make(T, 5, d, dt, 1, seed=13)
    v, S0, do, dST = ((x.float() * 1e30).to(x.dtype) for x in (v, S0, do, dST))
    o, ST = pace.pace_linattn_forward(q, k, v, g, S0=S0)
    check_forward(q, k, v, g, S0, cu, o, ST, dt)
    v, S0 = ((x.float() * 1e-30).to(x.dtype) for x in (v, S0))
    grads = pace.pace_linattn_backward(q, k, v, g, do, S0=S0, dST=dST)
    check_backward(q, k, v, g, S0, do, dST, cu, grads, dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_offsets_beyond_32_bits(dt):
    """Rows so far apart that the last ones lie more than 2^31 elements behind the first."""
    dt, T, H, d, far = DT[dt], 140, 1, 64, 1 << 24
    cu = np.array([0, 65, T])
    q, k, v, do, S0, dST = make(T, H, d, dt, 2, seed=14)
    g, dev_cu = torch.tensor([-0.02], device="cuda"), torch.from_numpy(cu.astype(np.int32)).cuda()
    room = torch.empty(T * far, device="cuda", dtype=dt).view(T, far)
    parts = [room[:, i * d:(i + 1) * d].unflatten(1, (H, d)) for i in range(8)]
    for x, y in zip(parts, (q, k, v, do)):
        x.copy_(y)
    o, ST = pace.pace_linattn_forward(*parts[:3], g, o=parts[4], cu_seqlens=dev_cu, max_len=75, S0=S0)
    check_forward(q, k, v, g, S0, cu, o, ST, dt)
    grads = pace.pace_linattn_backward(*parts[:3], g, parts[3], dq=parts[5], dk=parts[6], dv=parts[7], cu_seqlens=dev_cu,
                                       max_len=75, S0=S0, dST=dST)
    check_backward(q, k, v, g, S0, do, dST, cu, grads, dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_long_rows_at_odd_addresses(dt):
    """A long sequence whose rows are aligned to their elements only."""
    dt, T, H, d = DT[dt], 1300, 1, 64
    q, k, v, do, S0, dST = make(T, H, d, dt, 1, seed=9)
    g, cu = torch.tensor([-0.01], device="cuda"), np.array([0, T])

    def odd(x):
        y = torch.empty(x.numel() + 1, device="cuda", dtype=dt)[1:].view_as(x)
        return y.copy_(x)

    q1, k1, v1, do1 = (odd(x) for x in (q, k, v, do))
    o, ST = pace.pace_linattn_forward(q1, k1, v1, g, S0=S0)
    check_forward(q, k, v, g, S0, cu, o, ST, dt)
    grads = pace.pace_linattn_backward(q1, k1, v1, g, do1, S0=S0, dST=dST)
    check_backward(q, k, v, g, S0, do, dST, cu, grads, dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_two_graphs_and_an_eager_call(dt):
    """Two captured graphs, replayed in turn with eager calls between them, keep to their own workspaces."""
    dt, T, H, d = DT[dt], 2000, 1, 64
    g = decays(H)
    sets = [make(T, H, d, dt, 1, seed=s) for s in (1, 2, 3)]

    def all_of(q, k, v, do, S0, dST):
        return (pace.pace_linattn_forward(q, k, v, g, S0=S0) + pace.pace_linattn_backward(q, k, v, g, do, S0=S0, dST=dST))

    want = [all_of(*x) for x in sets]
    graphs, held = [], []
    for x in sets[:2]:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            held.append(all_of(*x))
    for _ in range(2):
        graphs[0].replay()
        eager = all_of(*sets[2])
        graphs[1].replay()
        graphs[0].replay()
    torch.cuda.synchronize()
    for a, b in zip(want, held + [eager]):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_a_layer_under_autograd():
    """Both directions as one autograd function, with shared key/value heads: the gradient of the shared heads is the
    sum over the query heads that read them."""
    n, T, H, d, dt = 2, 70, 4, 64, torch.float32

    class Retain(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, g):
            ctx.save_for_backward(q, k, v, g)
            return pace.pace_linattn_forward(q, k, v, g, num_seqs=n)[0]

        @staticmethod
        def backward(ctx, do):
            q, k, v, g = ctx.saved_tensors
            return (*pace.pace_linattn_backward(q, k, v, g, do.contiguous(), num_seqs=n)[:3], None)

    q, _, v, do, _, _ = make(n * T, H, d, dt, n, seed=6, states=False)
    k = make(n * T, 2, d, dt, n, seed=8, states=False)[1]
    g, cu = decays(H), np.arange(n + 1) * T
    for x in (q, k, v):
        x.requires_grad_()
    shared = k.repeat_interleave(2, 1)
    Retain.apply(q, shared, v, g).backward(do)
    (wq, bq), (wk, bk), (wv, bv), _ = ref.backward(f64(q), f64(shared), f64(v), f64(g), zeros(n, H, d), f64(do), zeros(n, H, d), cu)
    close(q.grad, wq, io_tol(bq, wq, dt, T, d))
    close(v.grad, wv, io_tol(bv, wv, dt, T, d))
    pair = lambda x: x.reshape(n * T, 2, 2, d).sum(2)  # noqa: E731
    close(k.grad, pair(wk), io_tol(pair(bk), pair(wk), dt, T, d) + ref.U32 * pair(bk))
