"""Which buffer a call gets that was given none: one for each stream, a new one under capture.
No GPU: the stream and its state are stand-ins, the buffers CPU memory."""
import pytest
import torch


@pytest.fixture
def so(monkeypatch):
    import __graft_entry__

    __graft_entry__._build_module().build()
    import cross_entropy_loss_gb300 as ce

    state = {"stream": 1, "capturing": False}
    monkeypatch.setattr(ce, "_stream_handle", lambda device, stream: state["stream"])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["capturing"])
    monkeypatch.setattr(ce, "_ws_cache", {})
    return ce, state


def test_a_stream_keeps_its_buffer_and_shares_it_with_none(so):
    ce, state = so
    a = ce.workspace(10, "cpu")
    assert a.numel() >= ce.foak_ce_workspace_size(10) and int(a.count_nonzero()) == 0
    assert ce.workspace(3, "cpu") is a
    state["stream"] = 2
    b = ce.workspace(10, "cpu")
    assert b.data_ptr() != a.data_ptr()
    more = ce.workspace(100_000, "cpu")  # this stream's grows, the other's stays
    assert more.numel() >= ce.foak_ce_workspace_size(100_000)
    assert ce.workspace(10, "cpu") is more
    state["stream"] = 1
    assert ce.workspace(10, "cpu") is a


def test_captured_calls_get_buffers_of_their_own(so):
    ce, state = so
    a = ce.workspace(10, "cpu")
    state["capturing"] = True
    b, c = ce.workspace(10, "cpu"), ce.workspace(10, "cpu")
    assert len({a.data_ptr(), b.data_ptr(), c.data_ptr()}) == 3
    assert int(b.count_nonzero()) == 0 and b.numel() >= ce.foak_ce_workspace_size(10)
    state["capturing"] = False
    assert ce.workspace(10, "cpu") is a


def test_a_workspace_of_another_device_is_refused(so):
    ce, _ = so
    ws = torch.zeros(4096, dtype=torch.uint8)
    assert ce._workspace_arg(ws, torch.device("cpu")) is ws
    with pytest.raises(ValueError):
        ce._workspace_arg(ws, torch.device("cuda", 0))
