"""The operators that sit between an LM head's logits and what a program does with them, with cases to time them on.

Five uses, all over the rows of an N x V logits matrix (bfloat16 or float32):

* ``logprobs``  the log probability of each row's given token, the entropy of its
  distribution and its K most likely tokens with their log probabilities (ties go to
  the lowest token id): a server answering with log probabilities, or a teacher whose
  top tokens are written down for a student;
* ``policy``    the same without the top tokens, then its backward pass from the
  gradients of the log probabilities and entropies: a policy-gradient step;
* ``distill``   the student's loss against a teacher's top tokens (mixed with the
  labels' cross-entropy) and its gradient in one call: a distillation step;
* ``distill2``  the same as a forward call and a backward call: the step under autograd;
* ``distill_eval``  the forward call alone: the loss on held-out data.

With z = x / T, p = softmax(z), T the temperature:

    logp = z_y - lse(z)     H = -sum_j p_j ln p_j
    dx_j = ([j = y] - p_j) g_logp / T - p_j (ln p_j + H) g_H / T
    q_k  = exp(t_k) / sum_l exp(t_l)   (the teacher's top K, renormalised; or exp(t_k) as it is)
    KD   = sum_k q_k (ln q_k - ln p_{id_k})        CE = lse(x) - x_y
    loss = sum over valid rows (ce_weight CE + kd_weight KD) / n_valid
    dx_j = (g / n_valid) (ce_weight (softmax(x)_j - [j = y])
                          + kd_weight / T (sum_k q_k p_j - sum_k q_k [j = id_k]))

Rows whose label is -100 are not valid: nothing is read of them, their outputs are zero
and their top ids -1.  A row in which every logit is -inf has lse -inf, log
probabilities -inf and entropy 0.
"""
import math

import torch

own = False

IGNORE = -100
GRAD_OUT = 0.25  # the loss's own gradient: one of four accumulated batches


def listed():
    return [
        # one token of a chat answer with its alternatives: latency
        dict(name="decode-1", op="logprobs", N=1, V=128256, dtype="bf16", K=20, T=1.0, ignored=0, mask="none"),
        # a serving batch of sampled tokens, some of them under a grammar that allows a handful of tokens
        dict(name="decode-64", op="logprobs", N=64, V=128256, dtype="bf16", K=20, T=0.7, ignored=0, mask="some"),
        # the log probabilities of a prompt batch at the framework's 4 x 1024 tokens of a 32000-token vocabulary
        dict(name="prompt-4096", op="logprobs", N=4096, V=32000, dtype="bf16", K=5, T=1.0, ignored=4, mask="none"),
        # a vocabulary of odd size, rows that do not start on a 16-byte boundary
        dict(name="prompt-odd", op="logprobs", N=777, V=50257, dtype="bf16", K=20, T=1.0, ignored=31, mask="some"),
        # a teacher in float32 writes down its top tokens at the distillation temperature
        dict(name="teacher-f32", op="logprobs", N=2048, V=128256, dtype="f32", K=64, T=2.0, ignored=100, mask="none"),
        # a teacher's pass over a packed batch
        dict(name="teacher-8192", op="logprobs", N=8192, V=128256, dtype="bf16", K=128, T=1.0, ignored=410, mask="none"),
        # a policy-gradient step on short answers
        dict(name="policy-256", op="policy", N=256, V=32000, dtype="f32", K=0, T=1.0, ignored=60, mask="none"),
        # a policy-gradient step on a long batch
        dict(name="policy-8192", op="policy", N=8192, V=128256, dtype="bf16", K=0, T=1.0, ignored=2000, mask="none"),
        # distillation mixed with the labels' loss at the framework's 4 x 1024 tokens
        dict(name="distill-4096", op="distill", N=4096, V=32000, dtype="bf16", K=64, T=2.0, ce=0.5, normalize=True, ignored=4, mask="none"),
        # pure distillation from a wide list at the 128256-token vocabulary
        dict(name="distill-8192", op="distill", N=8192, V=128256, dtype="bf16", K=128, T=1.0, ce=0.0, normalize=True, ignored=410, mask="none"),
        # the two-call form, odd vocabulary, the teacher's probabilities as they are
        dict(name="distill2-odd", op="distill2", N=515, V=49159, dtype="f32", K=50, T=1.0, ce=0.3, normalize=False, ignored=17, mask="none"),
        # a small held-out batch
        dict(name="eval-64", op="distill_eval", N=64, V=32000, dtype="bf16", K=16, T=1.5, ce=1.0, normalize=True, ignored=3, mask="none"),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "policy", "distill", "distill2", "distill_eval"])
    V = rng.choice([32000, 128256, 0, 0, 0]) or _between(rng, 8000, 160000)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    size = 2 if dtype == "bf16" else 4
    N = _between(rng, 1, min(8192, 8192 * 128256 * 2 // (V * size)))
    case = dict(op=op, N=N, V=V, dtype=dtype, K=0 if op == "policy" else _between(rng, 1, 128), T=rng.choice([1.0, 1.0, 0.7, 1.5, 2.0]),
                ignored=rng.randrange(0, N // 3 + 1), mask="none")
    if op == "logprobs":
        case["mask"] = rng.choice(["none", "none", "some"])
    if op.startswith("distill"):
        case["ce"] = rng.choice([0.0, 0.3, 0.5, 1.0])
        case["normalize"] = rng.choice([True, True, False])
    return case


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    N, V, K = case["N"], case["V"], case["K"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    # a broad body of logits, and a dozen likely tokens in each row
    x = torch.randn(N, V, generator=gen, device="cuda").mul_(2.0)
    apart = torch.randint(1, V // 13, (N, 1), generator=gen, device="cuda")
    hot = (torch.randint(0, V, (N, 1), generator=gen, device="cuda") + apart * torch.arange(12, device="cuda")) % V
    x.scatter_(1, hot, 6.0 + 6.0 * uniform(N, 12))
    drawn = torch.randint(0, V, (N,), generator=gen, device="cuda")
    labels = torch.where(uniform(N) < 0.7, hot[:, 0], drawn)
    order = torch.randperm(N, generator=gen, device="cuda")
    st = {"case": case}
    if case["mask"] == "some":
        # every third row allows seven tokens (its label among them), the next one every token but a quarter
        allowed = torch.zeros(N, V, dtype=torch.bool, device="cuda")
        allowed.scatter_(1, torch.cat([hot[:, :6], labels[:, None]], 1), True)
        kind = torch.arange(N, device="cuda") % 3
        quarter = uniform(N, V) < 0.25
        quarter.scatter_(1, labels[:, None], False)
        x.masked_fill_((kind[:, None] == 0) & ~allowed, -math.inf)
        x.masked_fill_((kind[:, None] == 1) & quarter, torch.finfo(dt).min)
        x.masked_fill_((order == N - 1)[:, None] & (N > 8), -math.inf)
    labels[order[: case["ignored"]]] = IGNORE
    st["labels"] = labels
    st["logits"] = x.to(dt, copy=True)
    if case["op"] == "policy":
        st["grad_logp"] = torch.randn(N, generator=gen, device="cuda") / N
        st["grad_entropy"] = torch.full((N,), -0.01 / N, device="cuda")
    if case["op"].startswith("distill"):
        # the teacher agrees with the student up to noise; some rows' last entries are padding
        z = x.add_(torch.randn(N, V, generator=gen, device="cuda")).div_(case["T"])
        top = z.topk(K, dim=1)
        st["teacher_logprobs"] = top.values - z.logsumexp(1, keepdim=True)
        ids = top.indices.to(torch.int32)
        short = (torch.arange(N, device="cuda") % 11 == 5)[:, None] & (torch.arange(K, device="cuda") >= (K + 1) // 2)[None, :]
        st["teacher_ids"] = ids.masked_fill_(short, -1)
        st["grad_out"] = torch.full((1,), GRAD_OUT, device="cuda")
    if case["op"] in ("policy", "distill", "distill2"):
        st["dlogits"] = torch.empty_like(st["logits"])
    return st


# ----------------------------------------------------------------- plain forms
def _valid(labels):
    return labels != IGNORE


def _softmax_parts(z, T):
    """Row maximum, (z - max) / T, its exponential and the sum of that, safe for rows of -inf alone."""
    m = z.amax(1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    d = (z - m) / T
    e = d.exp()
    return m, d, e, e.sum(1, keepdim=True)


def _plain_logprobs(x, labels, K, T):
    z = x.float()
    ok = _valid(labels)[:, None]
    m, d, e, s = _softmax_parts(z, T)
    ln_s = s.log()
    lse = m / T + ln_s
    y = labels.clamp(min=0)[:, None]
    logp = torch.where(s > 0, d.gather(1, y) - ln_s, lse)
    entropy = torch.where(s > 0, ln_s - torch.where(e > 0, e * d, 0.0).sum(1, keepdim=True) / s, 0.0)
    out = {"logp": torch.where(ok, logp, 0.0)[:, 0], "entropy": torch.where(ok, entropy, 0.0)[:, 0], "lse": torch.where(ok, lse, 0.0)[:, 0]}
    if K:
        # one whole number for each logit that orders by value, then by the lower token id
        bits = (z + 0.0).view(torch.int32)
        key = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long() << 32
        V = z.shape[1]
        key += torch.arange(V - 1, -1, -1, device=z.device)
        ids = V - 1 - (key.topk(K, dim=1).values & 0xFFFFFFFF)
        out["top_logprobs"] = torch.where(ok, torch.where(s > 0, d.gather(1, ids) - ln_s, lse), 0.0)
        out["top_ids"] = torch.where(ok, ids, -1).to(torch.int32)
    return out


def _plain_policy(x, labels, T, grad_logp, grad_entropy):
    z = x.float()
    ok = _valid(labels)[:, None]
    m, d, e, s = _softmax_parts(z, T)
    ln_s = s.log()
    y = labels.clamp(min=0)[:, None]
    logp = d.gather(1, y) - ln_s
    entropy = ln_s - torch.where(e > 0, e * d, 0.0).sum(1, keepdim=True) / s
    gl, gh = grad_logp[:, None], grad_entropy[:, None]
    p = e / s
    dx = -p * (gl + gh * (torch.where(p > 0, d - ln_s, 0.0) + entropy))
    dx.scatter_add_(1, y, gl)
    dx = torch.where(ok, dx / T, 0.0)
    return {"logp": torch.where(ok, logp, 0.0)[:, 0], "entropy": torch.where(ok, entropy, 0.0)[:, 0], "dlogits": dx.to(x.dtype)}


def _plain_distill(st, want_grad):
    case = st["case"]
    T, ce_w, kd_w = case["T"], case["ce"], 1.0 - 0.5 * case["ce"]
    z, labels = st["logits"].float(), st["labels"]
    ok = _valid(labels)[:, None]
    count = ok.sum()
    t = st["teacher_logprobs"].float()
    present = st["teacher_ids"] >= 0
    ids = st["teacher_ids"].clamp(min=0).long()
    y = labels.clamp(min=0)[:, None]
    q = torch.where(present, t, -math.inf).exp()
    if case["normalize"]:
        total = q.sum(1, keepdim=True)
        q = torch.where(total > 0, q / total, 0.0)
    m, d, e, s = _softmax_parts(z, T)
    lnp = d.gather(1, ids) - s.log()
    kd = torch.where(q > 0, q * (q.log() - lnp), 0.0).sum(1, keepdim=True)
    one = (z - m).exp()
    one_sum = one.sum(1, keepdim=True)
    ce = one_sum.log() - (z - m).gather(1, y)
    kd, ce = torch.where(ok, kd, 0.0), torch.where(ok, ce, 0.0)
    loss = ((ce_w * ce + kd_w * kd).double().sum() / count).float()
    out = {"loss": loss[None], "row_ce": ce[:, 0], "row_kd": kd[:, 0]}
    if want_grad:
        scale = GRAD_OUT / count
        dx = (scale * ce_w) * one / one_sum + (scale * kd_w / T) * q.sum(1, keepdim=True) * e / s
        dx.scatter_add_(1, ids, -(scale * kd_w / T) * q)
        dx.scatter_add_(1, y, (-scale * ce_w).expand(y.shape))
        out["dlogits"] = torch.where(ok, dx, 0.0).to(st["logits"].dtype)
    return out


def _plain(st):
    case = st["case"]
    if case["op"] == "logprobs":
        return _plain_logprobs(st["logits"], st["labels"], case["K"], case["T"])
    if case["op"] == "policy":
        return _plain_policy(st["logits"], st["labels"], case["T"], st["grad_logp"], st["grad_entropy"])
    out = _plain_distill(st, case["op"] != "distill_eval")
    return {k: v for k, v in out.items() if case["ce"] or k != "row_ce"}


# --------------------------------------------------------- the framework's calls
def _own(st):
    import cross_entropy_loss_gb300 as ce

    case, x, labels = st["case"], st["logits"], st["labels"]
    if case["op"] == "logprobs":
        r = ce.foak_logprobs_forward(x, labels, top_k=case["K"], temperature=case["T"], want_stats=False)
        return {k: r[k] for k in ("logp", "entropy", "lse", "top_logprobs", "top_ids")}
    if case["op"] == "policy":
        r = ce.foak_logprobs_forward(x, labels, temperature=case["T"], want_lse=False)
        dx, _ = ce.foak_logprobs_backward(x, labels, r["stats"], st["grad_logp"], r["entropy"], st["grad_entropy"], temperature=case["T"], dlogits=st["dlogits"])
        return {"logp": r["logp"], "entropy": r["entropy"], "dlogits": dx}
    how = dict(ce_weight=case["ce"], kd_weight=1.0 - 0.5 * case["ce"], temperature=case["T"], normalize=case["normalize"])
    ids, t = st["teacher_ids"], st["teacher_logprobs"]
    rows = ("row_ce", "row_kd") if case["ce"] else ("row_kd",)
    if case["op"] == "distill":
        r = ce.foak_distill_fwd_bwd(x, labels, ids, t, g=GRAD_OUT, dlogits=st["dlogits"], want_rows=True, **how)
        return {"loss": r["loss"], **{k: r[k] for k in rows}, "dlogits": r["dlogits"]}
    r = ce.foak_distill_forward(x, labels, ids, t, want_rows=True, want_stats=case["op"] == "distill2", **how)
    out = {"loss": r["loss"], **{k: r[k] for k in rows}}
    if case["op"] == "distill2":
        out["dlogits"], _ = ce.foak_distill_backward(x, labels, ids, t, r["stats"], st["grad_out"], dlogits=st["dlogits"], **how)
    return out


def run(st):
    return _own(st) if own else _plain(st)


def work(case):
    N, V, K = case["N"], case["V"], case["K"]
    rows = N - case["ignored"]
    size = 2 if case["dtype"] == "bf16" else 4
    read = rows * V * size
    # an exponential and three or four operations for each logit
    if case["op"] == "logprobs":
        return {"bytes": read + 8 * N + 12 * N + 8 * N * K, "flops": 5 * rows * V}
    if case["op"] == "policy":
        return {"bytes": 2 * read + N * V * size + 40 * N, "flops": 12 * rows * V}
    teacher = 8 * rows * K
    if case["op"] == "distill_eval":
        return {"bytes": read + teacher + 16 * N, "flops": 4 * rows * V}
    if case["op"] == "distill":
        return {"bytes": read + teacher + N * V * size + 16 * N, "flops": 8 * rows * V}
    return {"bytes": 2 * read + 2 * teacher + N * V * size + 40 * N, "flops": 8 * rows * V}


# ------------------------------------------------------------------- in 64 bits
def _lse64(z):
    top = z.max(dim=1).values.clamp(min=-1e308)
    return top + torch.exp(z - top[:, None]).sum(dim=1).log()


def exact(case, seed):
    st = prepare(case, seed)
    x, labels, T = st["logits"].double(), st["labels"], float(case["T"])
    rows = torch.arange(x.shape[0], device=x.device)
    keep = labels.ne(IGNORE)
    y = labels.masked_fill(~keep, 0)
    zero = torch.zeros((), dtype=torch.float64, device=x.device)
    if case["op"] in ("logprobs", "policy"):
        x /= T
        lse = _lse64(x)
        gone = torch.isinf(lse)  # nothing is left of such a row
        lnp = x - lse.masked_fill(gone, 0.0)[:, None]
        p = lnp.exp()
        entropy = -torch.xlogy(p, p).sum(dim=1)
        logp = lnp[rows, y]
        out = {"logp": logp.where(keep, zero), "entropy": entropy.where(keep, zero)}
        if case["op"] == "logprobs":
            out["lse"] = lse.where(keep, zero)
            if case["K"]:
                out["top_logprobs"] = lnp.topk(case["K"], dim=1).values.where(keep[:, None], zero)
                out["top_ids"] = None
            return out
        gl, gh = st["grad_logp"].double() / T, st["grad_entropy"].double() / T
        lnp.clamp_(min=-1e300)
        lnp += entropy[:, None]
        lnp *= gh[:, None]
        lnp += gl[:, None]
        dx = lnp.mul_(p).neg_()
        dx[rows, y] += gl
        dx[~keep] = 0.0
        out["dlogits"] = dx
        return out
    ce_w, kd_w, n = case["ce"], 1.0 - 0.5 * case["ce"], int(keep.sum())
    there = st["teacher_ids"].ge(0)
    ids = st["teacher_ids"].long().masked_fill(~there, 0)
    q = st["teacher_logprobs"].double().exp() * there
    if case["normalize"]:
        q = q / q.sum(dim=1, keepdim=True).clamp(min=1e-300)
    lse_t, lse_1 = _lse64(x / T), _lse64(x)
    kd = (torch.xlogy(q, q) - q * (x.gather(1, ids) / T - lse_t[:, None])).sum(dim=1).where(keep, zero)
    ce = (lse_1 - x[rows, y]).where(keep, zero)
    out = {"loss": ((ce_w * ce + kd_w * kd).sum() / n).reshape(1), "row_kd": kd}
    if ce_w:
        out["row_ce"] = ce
    if case["op"] != "distill_eval":
        grad = torch.exp(x / T - lse_t[:, None]) * (kd_w / T * q.sum(dim=1))[:, None]
        if ce_w:
            grad += ce_w * torch.exp(x - lse_1[:, None])
            grad[rows, y] -= ce_w
        flat = (rows[:, None] * x.shape[1] + ids).reshape(-1)
        grad.view(-1).index_add_(0, flat, (-kd_w / T * q).reshape(-1))
        grad *= GRAD_OUT / n
        grad[~keep] = 0.0
        out["dlogits"] = grad
    return out
