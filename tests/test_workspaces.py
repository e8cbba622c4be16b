"""CPU tests of the binding's default workspaces (no kernel is launched): which buffer a call gets."""

import threading

import pytest
import torch

import block_scaled_fp8_bfp8_amd as bfp8

HOST = torch.device("cpu")


@pytest.fixture
def state(monkeypatch):
    """A stand-in stream, and a switch for whether it is being captured."""
    s = {"capturing": False}
    monkeypatch.setattr(bfp8, "_stream", lambda device: 77)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: HOST.index)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: s["capturing"])
    return s


def test_a_captured_call_does_not_hold_the_kept_buffer(state):
    """A graph keeps the address of the buffer it was captured with. The kept one is replaced, and its memory given
    back, when a later call needs more; so a captured call may not have it, whether it was there before or not."""
    kept = bfp8._workspace(HOST, 4096)
    assert bfp8._workspace(HOST, 1024)[0] == kept[0]
    state["capturing"] = True
    captured = bfp8._workspace(HOST, 4096)
    assert captured[0] != kept[0] and captured[1] >= 4096
    state["capturing"] = False
    assert bfp8._workspace(HOST, 4096)[0] == kept[0]
    larger = bfp8._workspace(HOST, 8 << 20)
    state["capturing"] = True
    assert bfp8._workspace(HOST, 8 << 20)[0] != larger[0]


def test_nothing_is_made_where_nothing_is_needed(state):
    for state["capturing"] in (False, True):
        assert tuple(bfp8._workspace(HOST, 0))[:2] == (0, 0)


def test_host_threads_do_not_share_a_buffer(state):
    """A call of two launches uses its workspace in both; a second host thread's launches on the same stream may come
    between them."""
    mine = bfp8._workspace(HOST, 4096)
    got = []
    thread = threading.Thread(target=lambda: got.extend(bfp8._workspace(HOST, 4096) for _ in range(2)))
    thread.start()
    thread.join()
    assert got[0][0] == got[1][0] != mine[0]
    assert bfp8._workspace(HOST, 4096)[0] == mine[0]
