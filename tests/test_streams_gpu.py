"""Calls with a ``stream`` of their own: what they allocate is not shared with the caller's
stream while either may still use it."""
import pytest
import torch

import row_ops_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _calls(ce, N=96, V=5003, K=4):
    """Every row call as f(stream) -> outputs, on inputs that are complete."""
    x = ref.to_gpu(ref.make_logits(N, V, BF16, seed=1))
    y = torch.randint(0, V, (N,), generator=torch.Generator().manual_seed(1)).cuda()
    top = ce.foak_logprobs_forward(x, y, top_k=K)
    ids, t = top["top_ids"], top["top_logprobs"]
    lse = ce.foak_ce_forward(x, y)["lse"]
    ds = ce.foak_distill_forward(x, y, ids, t)
    gl = torch.ones(N, device="cuda")
    torch.cuda.synchronize()
    return {
        "logprobs_forward": lambda s: ce.foak_logprobs_forward(x, y, top_k=K, stream=s),
        "logprobs_backward": lambda s: ce.foak_logprobs_backward(x, y, top["stats"], gl, top["entropy"], gl, stream=s),
        "distill_forward": lambda s: ce.foak_distill_forward(x, y, ids, t, want_rows=True, stream=s),
        "distill_fwd_bwd": lambda s: ce.foak_distill_fwd_bwd(x, y, ids, t, want_rows=True, stream=s,
                                                             dlogits=torch.empty_like(x)),
        "distill_backward": lambda s: ce.foak_distill_backward(x, y, ids, t, ds["stats"], stream=s),
        "ce_forward": lambda s: ce.foak_ce_forward(x, y, want_row_loss=True, stream=s),
        "ce_backward": lambda s: ce.foak_ce_backward(x, y, lse, stream=s),
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
        assert torch.cuda.current_stream() == torch.cuda.default_stream()


def test_outputs_dropped_at_once_are_not_given_out_before_they_are_written(cuda_lib):
    side = torch.cuda.Stream()
    for name, call in _calls(cuda_lib).items():
        call(None)
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # the call's kernels are some 10 ms away
        sizes = [t.numel() * t.element_size() for t in _tensors(call(side))]  # dropped here
        keep = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
        torch.cuda.synchronize()
        assert all(bool((k == 0x5A).all()) for k in keep), name


def test_outputs_in_use_by_the_caller_are_not_given_out_to_the_stream(cuda_lib):
    """Dropped while the caller's stream has yet to read them: the stream's next call takes other memory."""
    ce = cuda_lib
    side = torch.cuda.Stream()
    call = _calls(ce)["distill_forward"]
    want = call(None)["row_kd"].clone()
    side.wait_stream(torch.cuda.current_stream())
    out = call(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(20_000_000)
    read = out["row_kd"].clone()
    sizes = [t.numel() * t.element_size() for t in _tensors(out)]
    del out
    with torch.cuda.stream(side):
        other = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    torch.cuda.synchronize()
    assert torch.equal(read, want) and len(other) > 0


def test_overlapping_calls_without_a_workspace(cuda_lib):
    """Two streams, calls of some 10 to 100 us each: losses, error words and the calls after them."""
    ce = cuda_lib
    N, V, K = 700, 32003, 8
    x = [ref.to_gpu(ref.make_logits(N, V, BF16, seed=i)) for i in range(2)]
    y = [torch.randint(0, V, (N,), generator=torch.Generator().manual_seed(i)).cuda() for i in range(2)]
    y[1][5] = V  # one of them reports a bad label
    top = [ce.foak_logprobs_forward(x[i], top_k=K) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]

    def step(i, stream):
        f = ce.foak_logprobs_forward(x[i], y[i], top_k=3, stream=stream)
        d = ce.foak_distill_forward(x[i], y[i], top[i]["top_ids"], top[i]["top_logprobs"], ce_weight=0.5, stream=stream)
        c = ce.foak_ce_forward(x[i], y[i], stream=stream)
        return [f["logp"], f["top_ids"], f["err"], d["loss"], d["n_valid"], d["err"], c["loss"], c["err"]]

    want = [[t.clone() for t in step(i, None)] for i in range(2)]
    assert [int(w[2]) for w in want] == [0, ce.FOAK_ERRBIT_LABEL_RANGE]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for i in range(2):
            got.append((i, step(i, streams[i])))
    torch.cuda.synchronize()
    got += [(i, step(i, None)) for i in range(2)]
    for i, outs in got:
        assert all(torch.equal(a, b) for a, b in zip(outs, want[i], strict=True))


def test_a_graph_has_a_workspace_of_its_own(cuda_lib):
    """Captured without one, after an eager call on the same stream whose buffer a larger call then
    replaces; replayed while eager calls run."""
    ce = cuda_lib
    N, V = 300, 32003
    x = ref.to_gpu(ref.make_logits(N, V, BF16, seed=3))
    y = torch.randint(0, V, (N,), generator=torch.Generator().manual_seed(3)).cuda()
    big = ref.to_gpu(ref.make_logits(5000, 130, BF16, seed=4))
    yb = torch.randint(0, 130, (5000,), generator=torch.Generator().manual_seed(4)).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        want = [ce.foak_logprobs_forward(x, y, top_k=5)["top_ids"].clone(), ce.foak_ce_forward(x, y)["loss"].clone()]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        a = ce.foak_logprobs_forward(x, y, top_k=5)
        b = ce.foak_ce_forward(x, y)
    with torch.cuda.stream(side):
        want_big = ce.foak_ce_forward(big, yb)["loss"].clone()
        other = torch.full((1 << 16,), 0x5A, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for _ in range(10):
        g.replay()
        with torch.cuda.stream(side):
            c = ce.foak_ce_forward(big, yb)
            d = ce.foak_logprobs_forward(x, y, top_k=5)
        torch.cuda.synchronize()
        assert torch.equal(a["top_ids"], want[0]) and torch.equal(b["loss"], want[1]) and int(a["err"]) == int(b["err"]) == 0
        assert torch.equal(c["loss"], want_big) and torch.equal(d["top_ids"], want[0])
    assert bool((other == 0x5A).all())


def test_a_workspace_in_host_memory_is_refused(cuda_lib):
    ce = cuda_lib
    x = torch.zeros(2, 8, device="cuda")
    ids, t = torch.zeros(2, 1, dtype=torch.int32, device="cuda"), torch.zeros(2, 1, device="cuda")
    for call in (lambda w: ce.foak_logprobs_forward(x, workspace_tensor=w),
                 lambda w: ce.foak_distill_forward(x, None, ids, t, workspace_tensor=w),
                 lambda w: ce.foak_distill_fwd_bwd(x, None, ids, t, workspace_tensor=w)):
        with pytest.raises(ValueError):
            call(torch.zeros(4096, dtype=torch.uint8))
        call(torch.zeros(4096, dtype=torch.uint8, device="cuda"))
