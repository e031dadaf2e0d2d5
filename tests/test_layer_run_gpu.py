"""Residual norms, rotary positions and the paged cache together, as a decoder layer's training and serving use
them; on streams of their own and in captured graphs."""
import threading

import pytest
import torch

import block_ops_ref as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _rotate64(x, pos, inv_freq):
    """Half layout, the whole head, in 64 bits: positions are small."""
    angle = pos.double()[:, None] * torch.tensor(inv_freq, dtype=torch.float64, device=x.device)
    co, si = angle.cos()[:, None], angle.sin()[:, None]
    a, b = x.chunk(2, dim=-1)
    return torch.cat([a * co - b * si, b * co + a * si], -1)


@pytest.mark.parametrize("post,gate", [(False, "none"), (True, "channel"), (True, "full"), (False, "row")])
def test_a_training_step(cuda_lib, post, gate):
    """Block output -> residual norm -> product -> rotary, and all the way back, against autograd in 64 bits.

    Six stages (two products, two norms' passes, two rotations) of sums of at most 128 terms: each within
    (128 + 86) U of its sum of absolute values, which for these random inputs is below ten times the result in the
    2-norm: 6 * 214 * 10 U = 7.7e-4.
    """
    ce, T, D, H, d = cuda_lib, 37, 128, 4, 16
    c = ref.make_norm(T, D, "f32", gate, post, seed=31)
    g = torch.Generator().manual_seed(7)
    W, out_grad, dH = torch.randn(D, H * d, generator=g) / D ** 0.5, torch.randn(T, H, d, generator=g), torch.randn(T, D, generator=g)
    pos = torch.arange(T) * 3
    plan = ce.foak_rotary_plan(d)
    x = {k: None if v is None else v.cuda() for k, v in c.items()}
    how = dict(gate=x["gate"], post_gamma=x["post_gamma"], scale=0.22)
    f = ce.foak_residual_norm_forward(x["X"], x["R"], x["gamma"], **how)
    q = (f["Y"] @ W.cuda()).view(T, H, d)
    turned, _ = ce.foak_rotary_apply(plan, pos.cuda(), q)
    dq, _ = ce.foak_rotary_apply(plan, pos.cuda(), out_grad.cuda(), inverse=True)
    dW, dY = f["Y"].t() @ dq.view(T, -1), dq.view(T, -1) @ W.cuda().t()
    b = ce.foak_residual_norm_backward(dY, dH.cuda(), f["H"], f["rstd"], x["gamma"], X=x["X"], post_rstd=f["post_rstd"], **how)

    t = {k: None if v is None else v.double().requires_grad_(k in ("X", "R", "gamma", "gate", "post_gamma")) for k, v in c.items()}
    W64 = W.double().requires_grad_(True)
    u = t["X"]
    if post:
        u = u * (u.square().mean(1, keepdim=True) + 1e-5).rsqrt() * t["post_gamma"]
    h = t["R"] + 0.22 * u * (1.0 if t["gate"] is None else t["gate"])
    y = h * (h.square().mean(1, keepdim=True) + 1e-5).rsqrt() * t["gamma"]
    z = _rotate64((y @ W64).view(T, H, d), pos, plan.inv_freq)
    ((z * out_grad.double()).sum() + (h * dH.double()).sum()).backward()
    want = {"dX": t["X"].grad, "dR": t["R"].grad, "dgamma": t["gamma"].grad}
    if gate != "none":
        want["dgate"] = t["gate"].grad
    if post:
        want["dpost_gamma"] = t["post_gamma"].grad
    got = {k: b[k] for k in want}
    got["dW"], want["dW"] = dW, W64.grad
    got["out"], want["out"] = turned, z.detach()
    for k, w in want.items():
        off = (got[k].cpu().double().reshape(w.shape) - w).norm()
        assert off <= 6 * 214 * 10 * ref.U * w.norm(), (k, float(off / w.norm()))


def _serve(ce, dtype, heads_first, layout_r, steps):
    """Chunks of prompts, then single tokens, through kv_slots and kv_append; every sequence's keys rotated at
    once beside, which has to be the same to the bit: an element's result depends on its token alone."""
    Hq, Hk, d, page, B, layers = 4, 2, 64, 8, 3, 2
    r, interleaved = layout_r
    plan = ce.foak_rotary_plan(r, base=10000.0, interleaved=interleaved)
    g = torch.Generator().manual_seed(5)
    total = torch.tensor([sum(s[b] for s in steps) for b in range(B)])
    most = int(-(-total.max() // page)) + 1
    pages = B * most + 2
    table = torch.randperm(pages, generator=g)[: B * most].view(B, most).to(torch.int32).cuda()
    shape = (pages, Hk, page, d) if heads_first else (pages, page, Hk, d)
    caches = [(torch.zeros(shape, dtype=dtype, device="cuda"), torch.zeros(shape, dtype=dtype, device="cuda")) for _ in range(layers)]
    full = [[tuple(torch.randn(int(total[b]), h, d, generator=g).to(dtype).cuda() for h in (Hq, Hk, Hk)) for b in range(B)] for _ in range(layers)]
    lens = torch.zeros(B, dtype=torch.int64)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for new in steps:
        starts = torch.tensor([0] + [sum(new[: i + 1]) for i in range(B)], dtype=torch.int32)
        T = int(starts[-1]) + 2
        at = ce.foak_kv_slots(table, lens.to(torch.int32).cuda(), starts.cuda(), T, page_size=page, num_pages=pages, err=err)
        for layer in range(layers):
            part = [torch.cat([full[layer][b][i][lens[b] : lens[b] + new[b]] for b in range(B)] + [torch.zeros(2, (Hq, Hk, Hk)[i], d, dtype=dtype, device="cuda")]) for i in range(3)]
            q = ce.foak_kv_append(part[1], part[2], *caches[layer], at["slots"], heads_first=heads_first, plan=plan, positions=at["positions"], q=part[0], err=err)
            for b in range(B):
                pos = torch.arange(int(lens[b]), int(lens[b]) + new[b], device="cuda")
                if new[b]:
                    alone, _ = ce.foak_rotary_apply(plan, pos, full[layer][b][0][lens[b] : lens[b] + new[b]])
                    assert torch.equal(q[int(starts[b]) : int(starts[b + 1])], alone)
        lens += torch.tensor(new)
    assert int(err) == 0
    for layer in range(layers):
        for b in range(B):
            n = int(total[b])
            want, _ = ce.foak_rotary_apply(plan, torch.arange(n, device="cuda"), full[layer][b][1])
            for cache, rows in zip(caches[layer], (want, full[layer][b][2])):
                seen = cache[table[b].long()]
                seen = seen.transpose(1, 2) if heads_first else seen
                assert torch.equal(seen.reshape(-1, Hk, d)[:n], rows)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("layout_r", [(64, False), (32, True)])
def test_serving(cuda_lib, dtype, heads_first, layout_r):
    _serve(cuda_lib, dtype, heads_first, layout_r, [(17, 0, 300), (5, 9, 0), (1, 1, 1), (1, 1, 1), (0, 1, 0), (1, 1, 1)])


def test_a_long_prompt_equals_its_tokens(cuda_lib):
    """Calls of every size take different ways through the kernels; the elements are the same."""
    ce = cuda_lib
    plan = ce.foak_rotary_plan(96, base=500000.0, scaling="bands", factor=8.0, original=8192.0)
    for dtype in (F32, BF16):
        q = torch.randn(6000, 12, 128, device="cuda").to(dtype)
        pos = torch.randint(0, 100000, (6000,), device="cuda")
        whole, _ = ce.foak_rotary_apply(plan, pos, q)
        for a, b in ((0, 1), (5, 8), (100, 900), (0, 3000)):
            part, _ = ce.foak_rotary_apply(plan, pos[a:b].contiguous(), q[a:b])
            assert torch.equal(part, whole[a:b])


def test_a_captured_step_of_a_padded_batch(cuda_lib):
    """One graph of fixed size, replayed for steps of fewer and fewer sequences."""
    ce = cuda_lib
    T, B, Hq, Hk, d, page, pages = 8, 8, 4, 2, 64, 4, 40
    plan = ce.foak_rotary_plan(d)
    table = torch.arange(B * 4, dtype=torch.int32, device="cuda").view(B, 4)
    lens, starts = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    q, k, v = (torch.randn(T, h, d, device="cuda") for h in (Hq, Hk, Hk))
    kc, vc = torch.zeros(pages, page, Hk, d, device="cuda"), torch.zeros(pages, page, Hk, d, device="cuda")
    X, R, gamma = torch.randn(T, 256, device="cuda"), torch.randn(T, 256, device="cuda"), torch.ones(256, device="cuda")
    q_out, err = torch.zeros_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")

    def step():
        f = ce.foak_residual_norm_forward(X, R, gamma)
        at = ce.foak_kv_slots(table, lens, starts, T, page_size=page, num_pages=pages, err=err)
        ce.foak_kv_append(k, v, kc, vc, at["slots"], plan=plan, positions=at["positions"], q=q, q_out=q_out, err=err)
        return f, at

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f, at = step()
    have = [0] * B
    for n in (8, 5, 1, 0):  # the first n sequences have a token each
        lens.copy_(torch.tensor(have, dtype=torch.int32))
        starts.copy_(torch.tensor([min(i, n) for i in range(B + 1)], dtype=torch.int32))
        for t in (q, k, v, X, R):
            t.normal_()
        q_out.fill_(3.0)
        before = kc.clone()
        graph.replay()
        torch.cuda.synchronize()
        want_slots = [table[b, have[b] // page].item() * page + have[b] % page for b in range(n)] + [-1] * (T - n)
        assert at["slots"].tolist() == want_slots and int(err) == 0
        assert bool((q_out[n:] == 3.0).all())
        want_q, want_k = ce.foak_rotary_apply(plan, at["positions"], q, k)
        assert torch.equal(q_out[:n], want_q[:n])
        flat, old = kc.view(-1, Hk, d), before.view(-1, Hk, d)
        rest = torch.ones(flat.shape[0], dtype=torch.bool, device="cuda")
        if n:
            where = torch.tensor(want_slots[:n], device="cuda")
            assert torch.equal(flat[where], want_k[:n]) and torch.equal(vc.view(-1, Hk, d)[where], v[:n])
            rest[where] = False
        assert torch.equal(flat[rest], old[rest])
        eager = ce.foak_residual_norm_forward(X, R, gamma)
        assert torch.equal(f["H"], eager["H"]) and torch.equal(f["Y"], eager["Y"])
        for b in range(n):
            have[b] += 1


def _calls(ce):
    """Every new call as f(stream) -> tensors, on inputs that are complete."""
    N, D, T = 900, 2048, 500
    c = {k: None if v is None else v.cuda() for k, v in ref.make_norm(N, D, "bf16", "channel", True, seed=2).items()}
    f = ce.foak_residual_norm_forward(c["X"], c["R"], c["gamma"], gate=c["gate"], post_gamma=c["post_gamma"])
    plan, pos = ce.foak_rotary_plan(128), torch.arange(T, device="cuda")
    q, k, v = (torch.randn(T, h, 128, device="cuda").bfloat16() for h in (8, 2, 2))
    table, lens, starts = torch.arange(64, dtype=torch.int32, device="cuda").view(1, 64), torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([0, T], dtype=torch.int32, device="cuda")
    at = ce.foak_kv_slots(table, lens, starts, T, page_size=16, num_pages=64)

    def append(s):
        kc, vc = (torch.zeros(64, 16, 2, 128, dtype=BF16, device="cuda") for _ in range(2))
        torch.cuda.synchronize()
        return ce.foak_kv_append(k, v, kc, vc, at["slots"], plan=plan, positions=at["positions"], q=q, stream=s), kc, vc

    torch.cuda.synchronize()
    return {
        "forward": lambda s: ce.foak_residual_norm_forward(c["X"], c["R"], c["gamma"], gate=c["gate"], post_gamma=c["post_gamma"], stream=s),
        "backward": lambda s: ce.foak_residual_norm_backward(c["dY"], c["dH"], f["H"], f["rstd"], c["gamma"], X=c["X"], gate=c["gate"], post_gamma=c["post_gamma"], post_rstd=f["post_rstd"], stream=s),
        "rotary": lambda s: ce.foak_rotary_apply(plan, pos, q, k, stream=s),
        "slots": lambda s: ce.foak_kv_slots(table, lens, starts, T, page_size=16, num_pages=64, stream=s),
        "append": append,
    }


def _tensors(out):
    return [t for t in (out.values() if isinstance(out, dict) else out) if t is not None]


def test_the_outputs_are_those_of_the_current_stream(cuda_lib):
    side = torch.cuda.Stream()
    for name, call in _calls(cuda_lib).items():
        a = _tensors(call(None))
        side.wait_stream(torch.cuda.current_stream())
        b = _tensors(call(side))
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        for i, (p, q) in enumerate(zip(a, b, strict=True)):
            assert torch.equal(p, q), (name, i)


def test_outputs_dropped_at_once_are_not_given_out_before_they_are_written(cuda_lib):
    side = torch.cuda.Stream()
    calls = _calls(cuda_lib)
    del calls["append"]  # waits for its caches
    for name, call in calls.items():
        call(None)
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # the call's kernels are some 10 ms away
        sizes = [t.numel() * t.element_size() for t in _tensors(call(side))]  # dropped here
        keep = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
        torch.cuda.synchronize()
        assert all(bool((k == 0x5A).all()) for k in keep), name


def test_a_plan_dropped_while_a_stream_uses_it(cuda_lib):
    ce = cuda_lib
    side = torch.cuda.Stream()
    q, pos = torch.randn(64, 4, 128, device="cuda"), torch.arange(64, device="cuda")
    want, _ = ce.foak_rotary_apply(ce.foak_rotary_plan(128), pos, q)
    torch.cuda.synchronize()
    plan = ce.foak_rotary_plan(128)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got, _ = ce.foak_rotary_apply(plan, pos, q, stream=side)
    del plan
    other = [torch.full((64,), 0x5A5A5A5A, dtype=torch.int64, device="cuda") for _ in range(16)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and len(other) == 16


def test_overlapping_backwards_and_graphs_have_workspaces_of_their_own(cuda_lib):
    """Two streams and two captured graphs, each with partial sums in flight."""
    ce = cuda_lib
    N, D = 3000, 1024
    cases = []
    for seed in range(2):
        c = {k: None if v is None else v.cuda() for k, v in ref.make_norm(N, D, "bf16", "channel", True, seed=seed).items()}
        f = ce.foak_residual_norm_forward(c["X"], c["R"], c["gamma"], gate=c["gate"], post_gamma=c["post_gamma"])
        cases.append((c, f))

    def back(i, stream=None):
        c, f = cases[i]
        b = ce.foak_residual_norm_backward(c["dY"], c["dH"], f["H"], f["rstd"], c["gamma"], X=c["X"], gate=c["gate"], post_gamma=c["post_gamma"], post_rstd=f["post_rstd"], stream=stream)
        return [b[k] for k in ("dR", "dX", "dgamma", "dgate", "dpost_gamma")]

    want = [[t.clone() for t in back(i)] for i in range(2)]
    torch.cuda.synchronize()
    streams, graphs, outs = [torch.cuda.Stream() for _ in range(2)], [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[i]):
            outs.append(back(i))
        graphs.append(g)
    got = []
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
            got.append((i, back(i, streams[1 - i])))
    torch.cuda.synchronize()
    for i, o in got + [(0, outs[0]), (1, outs[1])]:
        assert all(torch.equal(a, b) for a, b in zip(o, want[i], strict=True))


def test_backwards_of_two_host_threads_on_one_stream(cuda_lib):
    """Their launches do not come between one another's, whose partial sums lie in the stream's workspace."""
    ce = cuda_lib
    cases, want, wrong = [], [], [0, 0]
    for seed in range(2):
        c = {k: None if v is None else v.cuda() for k, v in ref.make_norm(400, 1024, "bf16", "none", True, seed=seed).items()}
        f = ce.foak_residual_norm_forward(c["X"], c["R"], c["gamma"], post_gamma=c["post_gamma"])
        cases.append((c, f))

    def back(i):
        c, f = cases[i]
        b = ce.foak_residual_norm_backward(c["dY"], c["dH"], f["H"], f["rstd"], c["gamma"], X=c["X"], post_gamma=c["post_gamma"], post_rstd=f["post_rstd"])
        return torch.cat([b["dgamma"], b["dpost_gamma"]])

    def many(i):
        for _ in range(20):
            outs = [back(i) for _ in range(50)]
            wrong[i] += sum(not torch.equal(o, want[i]) for o in outs)

    want.extend(back(i) for i in range(2))
    threads = [threading.Thread(target=many, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert wrong == [0, 0]


def test_the_shared_workspace_of_calls_in_a_row(cuda_lib):
    """Sizes that shrink and grow on one stream, with the cached workspace and with the caller's own."""
    ce = cuda_lib
    own = torch.empty(ce.foak_residual_norm_workspace_size(800, 8192), dtype=torch.uint8, device="cuda")
    for N, D in ((800, 512), (3, 8192), (800, 4096), (1, 64), (200, 8192)):
        c = ref.make_norm(N, D, "f32", "row", True, seed=N)
        f = ref.norm_forward(c["X"], c["R"], c["gamma"], c["gate"], c["post_gamma"], 1.0, 1e-5, 1e-5)
        rstd, post = f["rstd"][0].float(), f["post_rstd"][0].float()
        H = f["H"][0].float()
        want = ref.norm_backward(c["dY"], c["dH"], H, rstd, c["gamma"], c["X"], c["gate"], c["post_gamma"], post, 1.0)
        for ws in (None, own):
            b = ce.foak_residual_norm_backward(c["dY"].cuda(), c["dH"].cuda(), H.cuda(), rstd.cuda(), c["gamma"].cuda(), X=c["X"].cuda(), gate=c["gate"].cuda(), post_gamma=c["post_gamma"].cuda(), post_rstd=post.cuda(), workspace_tensor=ws)
            for k, w in want.items():
                ref.assert_close(b[k], w, (k, N, D))


def test_refused_under_the_synchronous_check(cuda_lib, monkeypatch):
    """FOAK_SYNC_CHECK turns the error word into a status."""
    ce = cuda_lib
    monkeypatch.setenv("FOAK_SYNC_CHECK", "1")
    kc, vc = torch.zeros(2, 4, 1, 16, device="cuda"), torch.zeros(2, 4, 1, 16, device="cuda")
    k, err = torch.ones(2, 1, 16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ce.foak_kv_append(k, k, kc, vc, torch.tensor([0, 7], device="cuda"), err=err)
    with pytest.raises(ce.FoakError) as e:
        ce.foak_kv_append(k, k, kc, vc, torch.tensor([0, 8], device="cuda"), err=err)
    assert e.value.status == ce.FOAK_ERR_PAGE_RANGE
