"""Where a call's own workspace comes from when it runs on another stream (on the host)."""
import contextlib

import torch

from zero_partitioned_mixed_adam_gb300 import ZERO_LINEAR_BACKWARD, train_ops


def test_the_workspace_is_of_the_calls_stream(monkeypatch):
    """PyTorch's allocator hands out memory that is free in the order of the stream that is
    current: the workspace is taken while the call's own stream is."""
    current = []

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    taken = []

    def empty(*args, real=torch.empty, **kw):
        taken.append(tuple(current))
        return real(*args, **kw)

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle))
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
    shape = train_ops.ZeroLinear(64, 128, 96)
    for given, want in ((None, ()), ("side", ("side",)), (4096, (("external", 4096),))):
        workspace, nbytes = train_ops._linear_workspace(shape, ZERO_LINEAR_BACKWARD, 2, 1, None, "cpu", given)
        assert nbytes == workspace.numel() > 0
        assert taken.pop() == want and not taken
