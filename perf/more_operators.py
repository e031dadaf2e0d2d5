"""The operators that a decoder layer needs around its matrix products, with cases to time them on.

Five uses:

* ``norm``       a block's output joins the residual stream and the next block's input is
  normalised: optional norm after the block, gate, residual scale, norm before the next block;
* ``norm_grad``  its backward pass from what the forward kept;
* ``rotary``     rotary positions on queries and keys: half and interleaved layouts, part of the head,
  frequencies scaled for long contexts; the forward, and with ``inverse`` the gradients' way back;
* ``append``     a serving step's tokens take their slots in a paged cache; keys are rotated into it,
  values copied, queries rotated beside it.

With X the block's output, R the residual stream, s the scale, g the gate ([D], [N, 1] or [N, D]):

    u = X, or X r1 post_gamma with r1 = 1 / sqrt(mean X^2 + eps)        h = R + s g u
    r = 1 / sqrt(mean h^2 + eps)                                        y = h r gamma
    dh = dH + r (gamma dY - h r mean(h r gamma dY))                     dR = dh
    dgamma = sum_i dY h r        dg = s dh u, summed where g was broadcast        du = s g dh
    dX = du, or r1 (post_gamma du - X r1 mean(X r1 post_gamma du)),     dpost_gamma = sum_i du X r1

Rotary: pair i of a head's first r elements, (i, i + r/2) or (2i, 2i + 1), turns by position times f_i and
is scaled by an attention factor c; f_i = base^(-2i/r), scaled as _frequencies says.

Token t of sequence b, the (t - start_b)-th of this step, has position cache_len_b + t - start_b and goes
to slot page_table[b][position / page_size] page_size + position mod page_size; rows behind the
last sequence are padding, with slot -1.
"""
import functools
import math

import torch

own = False

EPS = 1e-5


def listed():
    return [
        # one token of a chat answer between two blocks: latency
        dict(name="norm-decode-1", op="norm", N=1, D=4096, dtype="bf16", gate="none", post=False, scale=1.0),
        # a training batch of the framework's 8192 tokens, the block's output times a residual multiplier
        dict(name="norm-train-8192", op="norm", N=8192, D=4096, dtype="bf16", gate="none", post=False, scale=0.22),
        # norms on both sides of a block and an elementwise gate, odd sizes, in float32
        dict(name="norm-both-odd", op="norm", N=1537, D=5000, dtype="f32", gate="full", post=True, scale=1.0),
        # a wide model with one gate a channel
        dict(name="norm-wide", op="norm", N=2048, D=16384, dtype="bf16", gate="channel", post=False, scale=1.0),
        # the backward pass of norm-train-8192
        dict(name="grad-train-8192", op="norm_grad", N=8192, D=4096, dtype="bf16", gate="none", post=False, scale=0.22, stream=True),
        # the backward pass with norms on both sides and a gate a channel
        dict(name="grad-both-8192", op="norm_grad", N=8192, D=4096, dtype="bf16", gate="channel", post=True, scale=1.0, stream=True),
        # a short fine-tuning batch in float32, one gate a token, the last block (no gradient along the stream)
        dict(name="grad-row-f32", op="norm_grad", N=777, D=2056, dtype="f32", gate="row", post=False, scale=0.5, stream=False),
        # queries and keys of the framework's 8192 tokens with 32 + 8 heads, context extended by bands
        dict(name="rotary-8192", op="rotary", T=8192, Hq=32, Hk=8, d=128, r=128, layout="half", scaling="bands", dtype="bf16", inverse=False, far=131072),
        # gradients through an interleaved rotation of part of the head, in float32
        dict(name="rotary-part-grad", op="rotary", T=3001, Hq=20, Hk=4, d=80, r=32, layout="interleaved", scaling="none", dtype="f32", inverse=True, far=4096),
        # one token of a chat answer: latency
        dict(name="append-decode-1", op="append", B=1, most=1, context=2000, Hq=32, Hk=8, d=128, r=128, layout="half", scaling="bands", dtype="bf16", page=16, heads_first=False, padding=0),
        # a serving batch of one token each, in a padded graph batch, part of the head interleaved
        dict(name="append-decode-256", op="append", B=256, most=1, context=400, Hq=48, Hk=8, d=96, r=48, layout="interleaved", scaling="none", dtype="bf16", page=16, heads_first=True, padding=9),
        # chunks of several prompts
        dict(name="append-prompts", op="append", B=5, most=2500, context=3000, Hq=32, Hk=8, d=128, r=128, layout="half", scaling="ramp", dtype="bf16", page=64, heads_first=False, padding=40),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


MOST_BYTES = 400e6  # no drawn pass moves more than the largest listed one


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "norm_grad", "rotary", "rotary", "append", "append"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("norm"):
        D = 8 * _between(rng, 512 // 8, 16384 // 8)
        case = dict(op=op, N=1, D=D, dtype=dtype, gate=rng.choice(["none", "channel", "row", "full"]), post=rng.choice([False, True]), scale=rng.choice([1.0, 0.22, 0.5]))
        if op == "norm_grad":
            case["stream"] = rng.choice([True, True, False])
        row = work({**case, "N": 65})["bytes"] - work({**case, "N": 64})["bytes"]
        case["N"] = _between(rng, 1, min(16384, int(MOST_BYTES / row)))
        return case
    d = rng.choice([64, 80, 96, 128, 128, 192, 256])
    Hk = rng.choice([1, 2, 4, 8, 8, 16])
    case = dict(op=op, Hq=Hk * rng.choice([1, 2, 4, 5, 8]), Hk=Hk, d=d, r=rng.choice([d, d, d // 2, d // 4]), layout=rng.choice(["half", "interleaved"]), scaling=rng.choice(["none", "linear", "ntk", "bands", "ramp"]), dtype=dtype)
    heads = (case["Hq"] + 2 * Hk) * d * (2 if dtype == "bf16" else 4)
    if op == "rotary":
        case.update(T=_between(rng, 1, max(1, min(16384, int(MOST_BYTES / 4 / heads)))), inverse=rng.choice([False, True]), far=rng.choice([4096, 131072, 1048576]))
        return case
    page = rng.choice([1, 16, 16, 48, 64, 256])
    room = int(200e6 / (Hk * d * (2 if dtype == "bf16" else 4)))  # tokens of the cache
    B = _between(rng, 1, min(256, room // (2 * page)))
    most = rng.choice([1, 1, _between(rng, 2, 2048)])
    most = max(1, min(most, 8192 // B, room // B // 2, int(MOST_BYTES / 4 / heads) // B))
    context = _between(rng, 1, max(1, min(65536, room) // B - most - page))
    case.update(B=B, most=most, context=context, page=page, heads_first=rng.choice([False, True]), padding=rng.choice([0, 0, 3, 17]))
    return case


# ------------------------------------------------------------------------ inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _uniform(gen, *shape):
    return torch.rand(*shape, generator=gen, device="cuda")


def _gate(case, gen):
    N, D = case["N"], case["D"]
    if case["gate"] == "channel":
        return 0.3 + 0.1 * _normal(gen, D)
    if case["gate"] == "row":
        return _uniform(gen, N, 1)
    return _normal(gen, N, D).sigmoid_() if case["gate"] == "full" else None


def _prepare_norm(case, gen, st):
    N, D, dt = case["N"], case["D"], _dtype(case)
    # a residual stream whose channels differ in size, some of them by far; a block's output of order one
    size = (0.5 * _normal(gen, D)).exp_()
    size[:: max(1, D // 5)] *= 30.0
    R = (_normal(gen, N, D) * size).to(dt)
    X = _normal(gen, N, D).to(dt)
    gamma = (1.0 + 0.2 * _normal(gen, D)).to(dt)
    post_gamma = (1.0 + 0.2 * _normal(gen, D)).to(dt) if case["post"] else None
    gate = _gate(case, gen)
    gate = None if gate is None else gate.to(dt)
    st.update(X=X, gamma=gamma, post_gamma=post_gamma, gate=gate)
    if case["op"] == "norm":
        st.update(R=R, H=torch.empty_like(R), Y=torch.empty_like(R))
        return
    # what the forward left
    u = X.float()
    if case["post"]:
        st["post_rstd"] = (u.square().mean(1) + EPS).rsqrt()
        u = u * st["post_rstd"][:, None] * post_gamma.float()
    h = R.float() + case["scale"] * (u if gate is None else u * gate.float())
    st["rstd"] = (h.square().mean(1) + EPS).rsqrt()
    st["H"] = h.to(dt)
    st["dY"] = (_normal(gen, N, D) / 64).to(dt)
    st["dH"] = (_normal(gen, N, D) / 64).to(dt) if case["stream"] else None
    st.update(dR=torch.empty_like(R), dX=torch.empty_like(R))


def _prepare_heads(case, T, gen, st):
    # views of one product's output: queries, keys, values side by side
    Hq, Hk, d = case["Hq"], case["Hk"], case["d"]
    qkv = _normal(gen, T, Hq + 2 * Hk, d).to(_dtype(case))
    st.update(q=qkv[:, :Hq], k=qkv[:, Hq : Hq + Hk], v=qkv[:, Hq + Hk :])
    st["q_out"] = torch.zeros(T, Hq, d, dtype=qkv.dtype, device="cuda")


def _prepare_append(case, gen, st):
    B, page, Hk, d = case["B"], case["page"], case["Hk"], case["d"]
    new = torch.randint(max(1, case["most"] * 2 // 3), case["most"] + 1, (B,), generator=gen, device="cuda")
    lens = torch.randint(0, case["context"] + 1, (B,), generator=gen, device="cuda")
    starts = torch.zeros(B + 1, dtype=torch.int64, device="cuda")
    starts[1:] = new.cumsum(0)
    # as many rows and pages as the batch could need, whatever was drawn
    T = B * case["most"] + case["padding"]
    each = -(-(case["context"] + case["most"]) // page)
    pages = B * each + 3
    _prepare_heads(case, T, gen, st)
    st["page_table"] = torch.randperm(pages, generator=gen, device="cuda")[: B * each].view(B, each).to(torch.int32)
    st["cache_lens"], st["seq_starts"] = lens.to(torch.int32), starts.to(torch.int32)
    shape = (pages, Hk, page, d) if case["heads_first"] else (pages, page, Hk, d)
    st["k_cache"] = _normal(gen, *shape).to(_dtype(case))
    st["v_cache"] = _normal(gen, *shape).to(_dtype(case))
    st["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = {"case": case}
    if case["op"].startswith("norm"):
        _prepare_norm(case, gen, st)
    elif case["op"] == "rotary":
        _prepare_heads(case, case["T"], gen, st)
        # packed sequences: positions begin anew here and there, and reach far
        begin = torch.randint(0, case["far"], (1 + case["T"] // 512,), generator=gen, device="cuda")
        t = torch.arange(case["T"], device="cuda")
        st["positions"] = (begin[t // 512] + t % 512).contiguous()
        st["k_out"] = torch.zeros_like(st["k"], memory_format=torch.contiguous_format)
    else:
        _prepare_append(case, gen, st)
    return st


# ------------------------------------------------------------------- plain forms
BASE = 500000.0
FACTOR, LOW, HIGH, ORIGINAL = 8.0, 1.0, 4.0, 8192.0  # of the scaled contexts; "ramp" has 32 in the place of HIGH


def _frequencies(r, scaling, device):
    """(f_i in 64 bits, c): angle a position, and the factor of the rotated values."""
    i = torch.arange(r // 2, dtype=torch.float64, device=device)
    base = BASE * FACTOR ** (r / (r - 2)) if scaling == "ntk" else BASE
    f = torch.exp(i * (-2.0 * math.log(base) / r))
    if scaling == "linear":
        return f / FACTOR, 1.0
    if scaling == "bands":
        # by the turns that a frequency makes over the original context: below LOW stretched, above HIGH kept
        turns = ORIGINAL * f / (2.0 * math.pi)
        keep = ((turns - LOW) / (HIGH - LOW)).clamp(0.0, 1.0)
        return f * (keep + (1.0 - keep) / FACTOR), 1.0
    if scaling == "ramp":
        # the same by the frequency's index, between the whole indices of 32 turns and of one
        at = [r * math.log(ORIGINAL / (n * 2.0 * math.pi)) / (2.0 * math.log(BASE)) for n in (32.0, LOW)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), r - 1)
        stretch = ((i - lo) / (hi - lo if hi > lo else 0.001)).clamp(0.0, 1.0)
        return f * (1.0 - stretch + stretch / FACTOR), 0.1 * math.log(FACTOR) + 1.0
    return f, 1.0


def _plain_norm(st):
    case = st["case"]
    X, R, gate = st["X"].float(), st["R"].float(), st["gate"]
    u = X
    if case["post"]:
        u = X * (X.square().mean(1, keepdim=True) + EPS).rsqrt() * st["post_gamma"].float()
    h = R + case["scale"] * (u if gate is None else u * gate.float())
    y = h * (h.square().mean(1, keepdim=True) + EPS).rsqrt() * st["gamma"].float()
    return {"H": h.to(st["R"].dtype), "Y": y.to(st["R"].dtype)}


def _plain_norm_grad(st):
    case, dt = st["case"], st["X"].dtype
    s, gate, X = case["scale"], st["gate"], st["X"].float()
    r, dY = st["rstd"][:, None], st["dY"].float()
    hh = st["H"].float() * r
    t = st["gamma"].float() * dY
    dh = r * (t - hh * (hh * t).mean(1, keepdim=True))
    if case["stream"]:
        dh = dh + st["dH"].float()
    out = {"dR": dh.to(dt), "dgamma": (dY * hh).sum(0)}
    xh = X * st["post_rstd"][:, None] if case["post"] else X
    u = xh * st["post_gamma"].float() if case["post"] else X
    du = s * dh
    if case["gate"] == "channel":
        out["dgate"] = (du * u).sum(0)
    elif case["gate"] == "row":
        out["dgate"] = (du * u).sum(1, keepdim=True)
    elif case["gate"] == "full":
        out["dgate"] = (du * u).to(dt)
    if gate is not None:
        du = du * gate.float()
    if case["post"]:
        out["dpost_gamma"] = (du * xh).sum(0)
        v = st["post_gamma"].float() * du
        du = st["post_rstd"][:, None] * (v - xh * (xh * v).mean(1, keepdim=True))
    out["dX"] = du.to(dt)
    return out


def _plain_rotate(x, positions, case, inverse=False):
    r, half = case["r"], case["r"] // 2
    f, c = _frequencies(r, case["scaling"], x.device)
    theta = positions.double()[:, None] * f
    cos, sin = (theta.cos() * c).float()[:, None], (theta.sin() * c).float()[:, None]
    if inverse:
        sin = -sin
    z = x.float()
    out = z.clone()
    if case["layout"] == "half":
        a, b = z[..., :half], z[..., half:r]
        out[..., :half], out[..., half:r] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = z[..., 0:r:2], z[..., 1:r:2]
        out[..., 0:r:2], out[..., 1:r:2] = a * cos - b * sin, b * cos + a * sin
    return out.to(x.dtype)


def _plain_append(st):
    case, page = st["case"], st["case"]["page"]
    starts, lens = st["seq_starts"].long(), st["cache_lens"].long()
    t = torch.arange(st["q"].shape[0], device=starts.device)
    real = t < starts[-1]
    b = torch.where(real, (t[:, None] >= starts[None, 1:]).sum(1), 0)
    positions = torch.where(real, lens[b] + t - starts[b], 0)
    slots = torch.where(real, st["page_table"][b, positions // page].long() * page + positions % page, -1)
    rows = real.nonzero()[:, 0]
    at = slots[rows]
    k, v = _plain_rotate(st["k"], positions, case)[rows], st["v"][rows]
    if case["heads_first"]:
        st["k_cache"][at // page, :, at % page] = k
        st["v_cache"][at // page, :, at % page] = v
    else:
        st["k_cache"][at // page, at % page] = k
        st["v_cache"][at // page, at % page] = v
    st["q_out"][rows] = _plain_rotate(st["q"], positions, case)[rows]
    return {"slots": slots, "positions": positions, "q": st["q_out"], "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _plain(st):
    case = st["case"]
    if case["op"] == "norm":
        return _plain_norm(st)
    if case["op"] == "norm_grad":
        return _plain_norm_grad(st)
    if case["op"] == "rotary":
        return {n: _plain_rotate(st[n], st["positions"], case, case["inverse"]) for n in ("q", "k")}
    return _plain_append(st)


# ----------------------------------------------------------- the framework's calls
@functools.lru_cache(maxsize=None)
def _plan(r, layout, scaling):
    """A model's rotary plan: made once, from its configuration alone."""
    import cross_entropy_loss_gb300 as ce

    how = {} if scaling == "none" else dict(scaling=scaling, factor=FACTOR)
    if scaling in ("bands", "ramp"):
        how.update(low=LOW, high=HIGH if scaling == "bands" else 32.0, original=ORIGINAL)
    return ce.foak_rotary_plan(r, base=BASE, interleaved=layout == "interleaved", **how)


def _own(st):
    import cross_entropy_loss_gb300 as ce

    case = st["case"]
    if case["op"] == "norm":
        r = ce.foak_residual_norm_forward(st["X"], st["R"], st["gamma"], gate=st["gate"], post_gamma=st["post_gamma"], scale=case["scale"], eps=EPS, post_eps=EPS, H=st["H"], Y=st["Y"])
        return {"H": r["H"], "Y": r["Y"]}
    if case["op"] == "norm_grad":
        own_dX = case["post"] or case["gate"] != "none" or case["scale"] != 1.0  # otherwise it is dR
        r = ce.foak_residual_norm_backward(st["dY"], st["dH"], st["H"], st["rstd"], st["gamma"], X=st["X"], gate=st["gate"], post_gamma=st["post_gamma"], post_rstd=st.get("post_rstd"), scale=case["scale"], dR=st["dR"], dX=st["dX"] if own_dX else None)
        return {k: r[k] for k in ("dR", "dX", "dgamma", "dgate", "dpost_gamma") if r[k] is not None}
    plan = _plan(case["r"], case["layout"], case["scaling"])
    if case["op"] == "rotary":
        q, k = ce.foak_rotary_apply(plan, st["positions"], st["q"], st["k"], q_out=st["q_out"], k_out=st["k_out"], inverse=case["inverse"])
        return {"q": q, "k": k}
    at = ce.foak_kv_slots(st["page_table"], st["cache_lens"], st["seq_starts"], st["q"].shape[0], page_size=case["page"], num_pages=st["k_cache"].shape[0], err=st["err"])
    q = ce.foak_kv_append(st["k"], st["v"], st["k_cache"], st["v_cache"], at["slots"], heads_first=case["heads_first"], plan=plan, positions=at["positions"], q=st["q"], q_out=st["q_out"], err=st["err"])
    return {"slots": at["slots"], "positions": at["positions"], "q": q, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def run(st):
    return _own(st) if own else _plain(st)


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("norm"):
        N, D = case["N"], case["D"]
        n, full, post = N * D, case["gate"] == "full", case["post"]
        vectors = D * size * (1 + post + (case["gate"] == "channel")) + (N * size if case["gate"] == "row" else 0)
        if case["op"] == "norm":
            return {"bytes": (4 + full) * n * size + vectors, "flops": (9 + 4 * post) * n}
        # X is wanted where a norm or a gate stands on it; dX is its own where it is not dR
        reads = 2 + case["stream"] + (post or case["gate"] != "none") + full
        writes = 1 + (post or case["gate"] != "none" or case["scale"] != 1.0) + full
        grads = 4 * D * (1 + post + (case["gate"] == "channel")) + (4 * N if case["gate"] == "row" else 0)
        return {"bytes": (reads + writes) * n * size + vectors + grads + 4 * N * (1 + post), "flops": (14 + 10 * post) * n}
    Hq, Hk, d, r = case["Hq"], case["Hk"], case["d"], case["r"]
    if case["op"] == "rotary":
        T = case["T"]
        return {"bytes": 2 * T * (Hq + Hk) * d * size + 8 * T, "flops": 3 * T * (Hq + Hk) * r + 20 * T * r}
    # two thirds of the longest share is the least that a sequence brings: five sixths on the whole
    T = case["B"] * (max(1, case["most"] * 2 // 3) + case["most"]) // 2
    return {"bytes": 2 * T * (Hq + 2 * Hk) * d * size + 16 * (T + case["padding"]) + 16 * case["B"], "flops": 3 * T * (Hq + Hk) * r + 20 * T * r}


# -------------------------------------------------------------------- in 64 bits
def _exact_frequencies(r, scaling):
    out, base = [], BASE
    if scaling == "ntk":
        base = BASE * math.pow(FACTOR, r / (r - 2.0))
    first = math.floor(r * math.log(ORIGINAL / (64.0 * math.pi)) / math.log(BASE) / 2.0)
    last = math.ceil(r * math.log(ORIGINAL / (2.0 * math.pi * LOW)) / math.log(BASE) / 2.0)
    first, last = max(0, first), min(r - 1, last)
    for i in range(r // 2):
        f = math.pow(base, -2.0 * i / r)
        if scaling == "linear":
            f = f / FACTOR
        elif scaling == "bands":
            wave = 2.0 * math.pi / f
            if wave > ORIGINAL / LOW:
                f = f / FACTOR
            elif wave >= ORIGINAL / HIGH:
                w = (ORIGINAL / wave - LOW) / (HIGH - LOW)
                f = (1.0 - w) * f / FACTOR + w * f
        elif scaling == "ramp":
            w = min(1.0, max(0.0, (i - first) / (0.001 if first >= last else last - first)))
            f = f / FACTOR * w + f * (1.0 - w)
        out.append(f)
    return out, (1.0 + math.log(FACTOR) / 10.0 if scaling == "ramp" else 1.0)


def _exact_rotate(x, positions, case, sign):
    r = case["r"]
    f, c = _exact_frequencies(r, case["scaling"])
    angle = sign * positions.double()[:, None] * torch.tensor(f, dtype=torch.float64, device=x.device)
    turn = torch.polar(torch.full_like(angle, c), angle)[:, None]
    head, rest = x[..., :r].double(), x[..., r:].double()
    T, H, _ = x.shape
    pairs = head.reshape(T, H, r // 2, 2) if case["layout"] == "interleaved" else head.reshape(T, H, 2, r // 2).transpose(2, 3)
    done = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    done = done if case["layout"] == "interleaved" else done.transpose(2, 3)
    return torch.cat([done.reshape(T, H, r), rest], 2)


def _exact_norm(st, case):
    X, R, g = st["X"].double(), st["R"].double(), st["gamma"].double()
    if case["post"]:
        X = X / torch.sqrt(torch.sum(X * X, 1, True) / X.shape[1] + EPS) * st["post_gamma"].double()
    if st["gate"] is not None:
        X = X * st["gate"].double()
    h = torch.add(R, X, alpha=case["scale"])
    return {"H": h, "Y": h / torch.sqrt(torch.sum(h * h, 1, True) / h.shape[1] + EPS) * g}


def _exact_norm_grad(st, case):
    D, s = case["D"], case["scale"]
    dY, h, r = st["dY"].double(), st["H"].double(), st["rstd"].double().reshape(-1, 1)
    out = {"dgamma": torch.einsum("ij,ij,i->j", dY, h, r[:, 0])}
    t = dY * st["gamma"].double()
    dot = torch.einsum("ij,ij->i", t, h).reshape(-1, 1)
    dh = r * t - (r * r * r * dot / D) * h
    if st["dH"] is not None:
        dh = dh + st["dH"].double()
    out["dR"] = dh
    X, gate = st["X"].double(), st["gate"]
    g = torch.ones((), dtype=torch.float64, device=X.device) if gate is None else gate.double()
    if not case["post"]:
        out["dX"] = s * g * dh
        product = s * X * dh
    else:
        p, r1 = st["post_gamma"].double(), st["post_rstd"].double().reshape(-1, 1)
        product = s * r1 * p * X * dh
        v = s * g * p * dh
        out["dpost_gamma"] = (r1 * X * (s * g * dh)).sum(0)
        out["dX"] = r1 * v - r1 * r1 * r1 * X * ((X * v).sum(1, keepdim=True) / D)
    if gate is not None:
        out["dgate"] = product.sum(0) if case["gate"] == "channel" else product.sum(1, keepdim=True) if case["gate"] == "row" else product
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(st, case)
    if case["op"] == "norm_grad":
        return _exact_norm_grad(st, case)
    if case["op"] == "rotary":
        sign = -1.0 if case["inverse"] else 1.0
        return {n: _exact_rotate(st[n], st["positions"], case, sign) for n in ("q", "k")}
    # sequence by sequence, as the definition says
    page, starts, lens = case["page"], st["seq_starts"].tolist(), st["cache_lens"].tolist()
    table = st["page_table"].tolist()
    T = st["q"].shape[0]
    positions, slots = [0] * T, [-1] * T
    for b, begin in enumerate(starts[:-1]):
        for t in range(begin, starts[b + 1]):
            positions[t] = lens[b] + t - begin
            slots[t] = table[b][positions[t] // page] * page + positions[t] % page
    n = starts[-1]
    where = torch.tensor(positions, device="cuda")
    q = st["q_out"].double()
    q[:n] = _exact_rotate(st["q"][:n], where[:n], case, 1.0)
    to = torch.tensor(slots[:n], dtype=torch.int64, device="cuda")
    out = {"slots": None, "positions": None, "q": q}
    for name, rows in (("k_cache", _exact_rotate(st["k"][:n], where[:n], case, 1.0)), ("v_cache", st["v"][:n].double())):
        cache = st[name].double()
        flat = cache.transpose(1, 2).reshape(-1, case["Hk"], case["d"]) if case["heads_first"] else cache.reshape(-1, case["Hk"], case["d"])
        flat = flat.index_copy(0, to, rows)
        out[name] = flat.reshape(-1, page, case["Hk"], case["d"]).transpose(1, 2) if case["heads_first"] else flat.reshape(cache.shape)
    return out
