"""The cases on which two groups of operators are measured, in plain torch and in the library's kernels.

Linear attention with one fixed decay for each head (retention).  For head h with log decay g_h <= 0
    S_t = exp(g_h) S_{t-1} + v_t k_t^T,   o_t = S_t q_t,
  * "prompt": whole prompts, packed one behind the other, from a given or an empty state (chunked form);
  * "prompt_grad": its gradients for q, k, v and the initial state;
  * "token": one token for each sequence, the states updated in place (recurrent form).

Norms of queries and keys for each head and the position rotation in one pass ("norm", "norm_grad"):
    y = s R(pos) (w * x r),   r = (sum x^2 / n + eps)^(-1/2),   n = d (RMS) or 1 (L2),
R(pos) turns the pairs of the first `rot` channels by pos * inv_freq.  It makes the queries and keys of the above.

`own` chooses between the two: plain torch (False) and bit_recurrent_state_pace_b200 (True).
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_CHUNK = 64      # tokens a chunk of the plain form


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one user's next token through one layer of 32 heads: latency
        {"name": "token_1x32", "op": "token", "dtype": "bf16", "n": 1, "h": 32, "d": 128},
        # the next token of 256 sequences, 48 heads: the states fill 0.8 GB
        {"name": "token_256x48", "op": "token", "dtype": "bf16", "n": 256, "h": 48, "d": 128},
        # the exactness shape: two short prompts in fp32
        {"name": "prompt_tiny_f32", "op": "prompt", "dtype": "f32", "n": 2, "h": 2, "d": 32, "len": 16,
         "ragged": False, "state": True},
        # a serving batch of prompts of all lengths, some continuing from a stored state
        {"name": "prompt_ragged", "op": "prompt", "dtype": "bf16", "n": 64, "h": 32, "d": 128, "len": 1021,
         "ragged": True, "state": True},
        # one long document
        {"name": "prompt_long", "op": "prompt", "dtype": "bf16", "n": 1, "h": 32, "d": 128, "len": 32768,
         "ragged": False, "state": False},
        # small heads, lengths that end inside a chunk, in fp32
        {"name": "prompt_d64_f32", "op": "prompt", "dtype": "f32", "n": 8, "h": 16, "d": 64, "len": 1000,
         "ragged": False, "state": False},
        # a training micro-batch
        {"name": "grad_train", "op": "prompt_grad", "dtype": "bf16", "n": 8, "h": 32, "d": 128, "len": 4096,
         "ragged": False, "state": False},
        # packed training documents of uneven lengths, small heads, gradient through the states
        {"name": "grad_ragged_d64", "op": "prompt_grad", "dtype": "bf16", "n": 12, "h": 16, "d": 64, "len": 1500,
         "ragged": True, "state": True},
        # queries and keys of a decode batch (far positions)
        {"name": "norm_64_tokens", "op": "norm", "dtype": "bf16", "tokens": 64, "hq": 32, "hk": 32, "d": 128, "rot": 128,
         "pairs": "half", "kind": "rms", "weights": True, "far": True},
        # of long prompts, shared keys, a quarter of the channels turned
        {"name": "norm_prompt", "op": "norm", "dtype": "bf16", "tokens": 32768, "hq": 32, "hk": 8, "d": 128, "rot": 32,
         "pairs": "interleaved", "kind": "rms", "weights": True, "far": False},
        # of a training micro-batch
        {"name": "norm_grad_train", "op": "norm_grad", "dtype": "bf16", "tokens": 16384, "hq": 32, "hk": 32, "d": 128,
         "rot": 128, "pairs": "half", "kind": "rms", "weights": True, "far": False},
        # unit vectors in fp32, an odd number of tokens
        {"name": "norm_grad_l2_f32", "op": "norm_grad", "dtype": "f32", "tokens": 777, "hq": 16, "hk": 16, "d": 64,
         "rot": 64, "pairs": "half", "kind": "l2", "weights": False, "far": False},
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["token", "prompt", "prompt", "prompt_grad", "prompt_grad", "norm", "norm_grad"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "token":
        h = rng.choice([1, 4, 16, 31, 32, 48])
        return {"op": op, "dtype": dtype, "n": _spread(rng, 1, 12288 // h), "h": h, "d": rng.choice([32, 64, 128, 128])}
    if op in ("prompt", "prompt_grad"):
        h, d = rng.choice([1, 2, 7, 16, 32]), rng.choice([32, 64, 64, 128, 128])
        length = _spread(rng, 1, 16384)
        n = _spread(rng, 1, max(1, min(64, (1 << 19) // (h * length))))
        return {"op": op, "dtype": dtype, "n": n, "h": h, "d": d, "len": length, "ragged": rng.random() < 0.6,
                "state": rng.random() < 0.5}
    d = rng.choice([32, 64, 128, 128, 256])
    return {"op": op, "dtype": dtype, "tokens": _spread(rng, 1, 8192), "hq": rng.choice([1, 5, 16, 32]),
            "hk": rng.choice([1, 2, 8, 32]), "d": d, "rot": rng.choice([0, d // 4, d // 2, d]),
            "pairs": rng.choice(["half", "interleaved"]), "kind": rng.choice(["rms", "l2"]),
            "weights": rng.random() < 0.6, "far": rng.random() < 0.4}


def _lengths(case):
    """The prompts' lengths: all `len`, or uneven ones up to it (one of them `len`, one empty where there are four or more)."""
    n, most = case["n"], case["len"]
    if not case["ragged"]:
        return [most] * n
    r = random.Random(n * 1000003 + most)
    lens = [_spread(r, 1, most) for _ in range(n)]
    lens[r.randrange(n)] = most
    if n >= 4:
        lens[(lens.index(most) + 1) % n] = 0
    return lens


def work(case):
    e, d = (2 if case["dtype"] == "bf16" else 4), case["d"]
    if case["op"] == "token":
        heads = case["n"] * case["h"]
        return {"bytes": heads * (8 * d * d + 4 * d * e), "flops": heads * 5 * d * d}
    if case["op"] in ("prompt", "prompt_grad"):
        th, heads = sum(_lengths(case)) * case["h"], case["n"] * case["h"]
        grad = case["op"] == "prompt_grad"
        states = (3 if grad else 2) if case["state"] else (0 if grad else 1)
        return {"bytes": th * d * e * (7 if grad else 4) + heads * d * d * 4 * states, "flops": th * d * d * (10 if grad else 4)}
    values = case["tokens"] * (case["hq"] + case["hk"]) * d
    if case["op"] == "norm":
        return {"bytes": values * 2 * e + 4 * case["tokens"], "flops": values * 7}
    return {"bytes": values * 3 * e + 4 * case["tokens"], "flops": values * 16}


# ----------------------------------------------------------------------------------------------- inputs

def _log_decay(h):
    """The heads' log decays: -2^(-8 (i + 1) / h), from fast forgetting to a memory of hundreds of tokens."""
    i = torch.arange(1, h + 1, dtype=torch.float64)
    return (-torch.exp2(-8.0 * i / h)).float().cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt, d = _DT[case["dtype"]], case["d"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)

    def unit(*shape):          # queries and keys come normalised for each head
        x = normal(*shape)
        return (x / x.square().sum(-1, keepdim=True).add(1e-6).sqrt()).to(dt)

    def value(*shape):         # a few channels of the values are large
        x = normal(*shape)
        x[..., 3::32] *= 8.0
        return x.to(dt)

    st = {"case": dict(case)}
    if case["op"] == "token":
        n, h = case["n"], case["h"]
        st.update(q=unit(n, h, d), k=unit(n, h, d), v=value(n, h, d), g=_log_decay(h), S=normal(n, h, d, d))
        return st
    if case["op"] in ("prompt", "prompt_grad"):
        lens, h, n = _lengths(case), case["h"], case["n"]
        total = sum(lens)
        st.update(q=unit(total, h, d), k=unit(total, h, d), v=value(total, h, d), g=_log_decay(h), cu=None, S0=None)
        if case["ragged"]:
            st["cu"] = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()
        if case["state"]:
            st["S0"] = normal(n, h, d, d)
        if case["op"] == "prompt_grad":
            st["do"] = normal(total, h, d).to(dt)
            st["dST"] = normal(n, h, d, d) if case["state"] else None
        return st
    t, hq, hk, rot = case["tokens"], case["hq"], case["hk"], case["rot"]
    st.update(q=normal(t, hq, d).to(dt), k=(3.0 * normal(t, hk, d)).to(dt), wq=None, wk=None, pos=None, inv=None)
    if case["weights"]:
        st.update(wq=1.0 + 0.2 * normal(d), wk=1.0 + 0.2 * normal(d))
    if rot:
        i = torch.arange(rot // 2, dtype=torch.float64)
        st["inv"] = torch.pow(torch.tensor(1e4, dtype=torch.float64), -2.0 * i / rot).float().cuda()
        if case["far"]:
            st["pos"] = torch.randint(0, 1 << 20, (t,), generator=gen, device="cuda", dtype=torch.int32)
        else:
            first = torch.randint(0, 4096, (1,), generator=gen, device="cuda", dtype=torch.int32)
            st["pos"] = first + torch.arange(t, device="cuda", dtype=torch.int32)
    if case["op"] == "norm_grad":
        st.update(dq=normal(t, hq, d).to(dt), dk=normal(t, hk, d).to(dt))
    return st


_EPS = 1e-6


def _q_scale(case):
    return case["d"] ** -0.5


# ------------------------------------------------------------------------------------------ plain forms

def _padded_index(st, case):
    """[n, most] rows of the packed tokens, and whether there is one; `most` a multiple of the chunk."""
    most = -(-case["len"] // _CHUNK) * _CHUNK
    at = torch.arange(most, device="cuda")
    if st["cu"] is None:
        begin = torch.arange(case["n"], device="cuda") * case["len"]
        lens = torch.full((case["n"],), case["len"], device="cuda")
    else:
        begin, lens = st["cu"][:-1].long(), (st["cu"][1:] - st["cu"][:-1]).long()
    there = at[None, :] < lens[:, None]
    return torch.where(there, begin[:, None] + at[None, :], 0), there, lens


def _decayed(query, key, value, g, lens, S, back):
    """out_i = (sum_{j <= i} e^{g (i - j)} value_j key_j^T + e^{g i'} S) query_i in chunks, and the state behind the last token.

    query, key, value: fp32 [n, h, L, d], zero behind each sequence's end; S: fp32 [n, h, d, d] or None.
    Forwards i' = i + 1.  `back` runs from the last token to the first with i' the number of tokens behind i
    (S then is the gradient that reaches the last state)."""
    n, h, L, d = query.shape
    c, m = _CHUNK, L // _CHUNK
    t = torch.arange(c, device="cuda", dtype=torch.float32)
    cm = torch.arange(m + 1, device="cuda", dtype=torch.float32)
    gh, ln = g[:, None, None], lens.float()
    # within a chunk
    ages = (t[None, :] - t[:, None]) if back else (t[:, None] - t[None, :])          # [i, j]
    near = torch.where(ages >= 0, torch.exp(gh * ages.clamp(min=0)), 0.0)            # [h, c, c]
    q4, k4, v4 = (x.view(n, h, m, c, d) for x in (query, key, value))
    inner = torch.matmul(torch.matmul(q4, k4.transpose(-1, -2)) * near[None, :, None], v4)
    # each chunk's own contribution to the state at its far edge, and the state at every edge by a product over chunks
    edge = torch.exp(gh * (t + 1 if back else c - 1 - t)[None, :, None])             # [h, c, 1]
    U = torch.matmul((v4 * edge[None, :, None]).transpose(-1, -2), k4)               # [n, h, m, d, d]
    between = (cm[None, :-1] - cm[:, None]) if back else (cm[:, None] - 1 - cm[None, :-1])    # [edge, chunk]
    link = torch.where(between >= 0, torch.exp(gh * c * between.clamp(min=0)), 0.0)
    states = torch.matmul(link[None], U.reshape(n, h, m, d * d)).view(n, h, m + 1, d, d)
    if S is not None:
        tokens = (ln[:, None] - cm * c).clamp(min=0) if back else (cm * c).expand(n, m + 1)
        states = states + torch.exp(g[None, :, None] * tokens[:, None, :])[..., None, None] * S[:, :, None]
    if back:                                       # from a chunk's far edge over the tokens that are there behind i
        left = (ln[:, None, None] - 1 - (cm[:-1, None] * c + t)[None]).clamp(min=0)
        carry = torch.exp(g[None, :, None, None] * torch.minimum(left, c - 1 - t)[:, None])
        out = inner + carry[..., None] * torch.matmul(q4, states[:, :, 1:].transpose(-1, -2))
        return out.view(n, h, L, d), states[:, :, 0]
    carry = torch.exp(gh * (t + 1))[None, ..., None]                                 # [1, h, 1, c, 1]
    out = inner + carry * torch.matmul(q4, states[:, :, :-1].transpose(-1, -2))
    # the state behind the last token: the near edge of its chunk, and what the chunk's tokens bring
    row, last = torch.arange(n, device="cuda"), (lens - 1).clamp(min=0) // c
    age = (ln - 1 - last * c)[:, None, None] - t
    w = torch.where(age >= 0, torch.exp(gh[None, :, 0] * age.clamp(min=0)), 0.0)     # [n, h, c]
    end = torch.matmul((v4[row, :, last] * w[..., None]).transpose(-1, -2), k4[row, :, last])
    return out.view(n, h, L, d), end + torch.exp(g * (ln - last * c)[:, None])[..., None, None] * states[row, :, last]


def _prompt_plain(st, case):
    index, there, lens = _padded_index(st, case)
    total, h, d = st["q"].shape

    def padded(x):
        if total == 0:
            return torch.zeros(*index.shape, h, d, device="cuda").permute(0, 2, 1, 3)
        return torch.where(there[..., None, None], x[index].float(), 0.0).permute(0, 2, 1, 3).contiguous()

    def packed(x, like):
        out = torch.empty_like(like)
        out[index[there]] = x.permute(0, 2, 1, 3)[there].to(like.dtype)
        return out

    q, k, v, g, S0 = padded(st["q"]), padded(st["k"]), padded(st["v"]), st["g"], st["S0"]
    if case["op"] == "prompt":
        o, end = _decayed(q, k, v, g, lens, S0, False)
        return packed(o, st["q"]), end
    do = padded(st["do"])
    dq, _ = _decayed(do, v, k, g, lens, None if S0 is None else S0.transpose(-1, -2), False)
    dv, dS0 = _decayed(k, q, do, g, lens, st["dST"], True)
    dk, _ = _decayed(v, do, q, g, lens, None if st["dST"] is None else st["dST"].transpose(-1, -2), True)
    out = [packed(dq, st["q"]), packed(dk, st["k"]), packed(dv, st["v"])]
    return (*out, dS0) if case["state"] else tuple(out)


def _token_plain(st, case):
    S, q, k, v = st["S"], st["q"].float(), st["k"].float(), st["v"].float()
    S.mul_(torch.exp(st["g"])[None, :, None, None])
    S.add_(v[..., :, None] * k[..., None, :])
    return (S * q[..., None, :]).sum(-1).to(st["q"].dtype), S


def _turn(x, cos, sin, rot, pairs):
    """Turns the pairs of the first `rot` channels; cos, sin: [t, 1, rot / 2]."""
    y = x.clone()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if pairs == "interleaved" else (x[..., :rot // 2], x[..., rot // 2:rot])
    ya, yb = a * cos - b * sin, b * cos + a * sin
    if pairs == "interleaved":
        y[..., 0:rot:2], y[..., 1:rot:2] = ya, yb
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = ya, yb
    return y


def _norm_plain(st, case):
    rot, pairs, d = case["rot"], case["pairs"], case["d"]
    cos = sin = None
    if rot:                               # angles in 64 bits: positions reach a million
        angle = st["pos"].double()[:, None, None] * st["inv"].double()
        cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    width = float(d) if case["kind"] == "rms" else 1.0

    def one(x, w, scale):
        x = x.float()
        hat = x * torch.rsqrt(x.square().sum(-1, keepdim=True) / width + _EPS)
        y = hat * w if w is not None else hat
        return (_turn(y, cos, sin, rot, pairs) if rot else y) * scale

    def grad(x, w, dy, scale):
        x, u = x.float(), dy.float() * scale
        if rot:
            u = _turn(u, cos, -sin, rot, pairs)
        r = torch.rsqrt(x.square().sum(-1, keepdim=True) / width + _EPS)
        hat = x * r
        dw = (u * hat).sum((0, 1))
        dh = u * w if w is not None else u
        dx = r * (dh - hat * ((hat * dh).sum(-1, keepdim=True) / width))
        return dx, dw

    s, dt = _q_scale(case), st["q"].dtype
    if case["op"] == "norm":
        return one(st["q"], st["wq"], s).to(dt), one(st["k"], st["wk"], 1.0).to(dt)
    dq, dwq = grad(st["q"], st["wq"], st["dq"], s)
    dk, dwk = grad(st["k"], st["wk"], st["dk"], 1.0)
    out = [dq.to(dt), dk.to(dt)]
    return (*out, dwq, dwk) if case["weights"] else tuple(out)


# -------------------------------------------------------------------------------------------------- run

def _run_own(st, case):
    import bit_recurrent_state_pace_b200 as pace

    if case["op"] == "token":
        return pace.pace_linattn_step(st["S"], st["q"], st["k"], st["v"], st["g"]), st["S"]
    if case["op"] == "prompt":
        return pace.pace_linattn_forward(st["q"], st["k"], st["v"], st["g"], num_seqs=case["n"], max_len=case["len"],
                                         cu_seqlens=st["cu"], S0=st["S0"])
    if case["op"] == "prompt_grad":
        dq, dk, dv, dS0 = pace.pace_linattn_backward(
            st["q"], st["k"], st["v"], st["g"], st["do"], num_seqs=case["n"], max_len=case["len"],
            cu_seqlens=st["cu"], S0=st["S0"], dST=st["dST"], need_dS0=case["state"])
        return (dq, dk, dv, dS0) if case["state"] else (dq, dk, dv)
    how = dict(rotary_dim=case["rot"], interleaved=case["pairs"] == "interleaved", norm=case["kind"], eps=_EPS,
               q_scale=_q_scale(case))
    if case["op"] == "norm":
        return pace.pace_qk_norm_rotate(st["q"], st["k"], st["wq"], st["wk"], st["pos"], st["inv"], **how)
    dq, dk, dwq, dwk = pace.pace_qk_norm_rotate_backward(st["q"], st["k"], st["wq"], st["wk"], st["pos"], st["inv"],
                                                         st["dq"], st["dk"], **how)
    return (dq, dk, dwq, dwk) if case["weights"] else (dq, dk)


def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    if case["op"] == "token":
        return _token_plain(state, case)
    return _prompt_plain(state, case) if case["op"].startswith("prompt") else _norm_plain(state, case)


# ------------------------------------------------------------------------------------------------ exact

def _exact_prompt(case, st):
    """Token by token, all sequences side by side, from the recurrence itself in 64 bits."""
    lens, n, h, d = _lengths(case), case["n"], case["h"], case["d"]
    a = torch.exp(st["g"].double())[None, :, None, None]
    begin = torch.tensor([sum(lens[:i]) for i in range(n)], device="cuda")
    ends = torch.tensor(lens, device="cuda")
    q, k, v = st["q"].double(), st["k"].double(), st["v"].double()
    S = torch.zeros(n, h, d, d, dtype=torch.float64, device="cuda") if st["S0"] is None else st["S0"].double()
    o, grad = torch.zeros_like(q), case["op"] == "prompt_grad"
    do = st["do"].double() if grad else None
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q)
    order = sorted(range(n), key=lambda i: -lens[i])
    rank = torch.tensor(order, device="cuda")
    begin, ends, S = begin[rank], ends[rank], S[rank].clone()
    sizes = [lens[i] for i in order]
    most = sizes[0] if sizes else 0
    live = [sum(1 for x in sizes if x > t) for t in range(most)]
    for t in range(most):
        m = live[t]
        row = begin[:m] + t
        S[:m] = a * S[:m] + v[row].unsqueeze(-1) * k[row].unsqueeze(-2)
        if grad:
            dq[row] = torch.matmul(do[row].unsqueeze(-2), S[:m]).squeeze(-2)
        else:
            o[row] = torch.matmul(S[:m], q[row].unsqueeze(-1)).squeeze(-1)
    back = torch.argsort(rank)
    if not grad:
        return o, S[back]
    X = torch.zeros_like(S) if st["dST"] is None else st["dST"].double()[rank].clone()
    for t in reversed(range(most)):
        m = live[t]
        row = begin[:m] + t
        D = X[:m] + do[row].unsqueeze(-1) * q[row].unsqueeze(-2)
        dv[row] = torch.matmul(D, k[row].unsqueeze(-1)).squeeze(-1)
        dk[row] = torch.matmul(v[row].unsqueeze(-2), D).squeeze(-2)
        X[:m] = a * D
    return (dq, dk, dv, X[back]) if case["state"] else (dq, dk, dv)


def _exact_norm(case, st):
    """Pairs of channels as complex numbers; the gradients by differentiating that."""
    rot, d = case["rot"], case["d"]

    def rotated(y):
        if not rot:
            return y
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                           st["pos"].double()[:, None, None] * st["inv"].double())
        head, rest = y[..., :rot], y[..., rot:]
        if case["pairs"] == "interleaved":
            z = torch.complex(head.unflatten(-1, (rot // 2, 2))[..., 0], head.unflatten(-1, (rot // 2, 2))[..., 1]) * turn
            head = torch.stack([z.real, z.imag], -1).flatten(-2)
        else:
            z = torch.complex(*head.chunk(2, -1)) * turn
            head = torch.cat([z.real, z.imag], -1)
        return torch.cat([head, rest], -1)

    def forward(x, w, scale):
        size = x.pow(2).mean(-1, keepdim=True) if case["kind"] == "rms" else x.pow(2).sum(-1, keepdim=True)
        y = x / (size + _EPS).sqrt()
        return scale * rotated(y if w is None else y * w)

    wide = [(st["q"], st["wq"], st.get("dq"), _q_scale(case)), (st["k"], st["wk"], st.get("dk"), 1.0)]
    if case["op"] == "norm":
        return tuple(forward(x.double(), None if w is None else w.double(), s) for x, w, _, s in wide)
    dx, dw = [], []
    for x, w, dy, s in wide:
        leaf = x.double().requires_grad_()
        weight = None if w is None else w.double().requires_grad_()
        got = torch.autograd.grad(forward(leaf, weight, s), [leaf] + ([] if w is None else [weight]), dy.double())
        dx.append(got[0])
        dw += list(got[1:])
    return tuple(dx + dw)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "token":
        S = torch.exp(st["g"].double())[:, None, None] * st["S"].double()
        S += torch.einsum("nhi,nhj->nhij", st["v"].double(), st["k"].double())
        return torch.einsum("nhij,nhj->nhi", S, st["q"].double()), S
    return _exact_prompt(case, st) if case["op"].startswith("prompt") else _exact_norm(case, st)
