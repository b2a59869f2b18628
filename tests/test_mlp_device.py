"""The feed-forward layer's passes run with its tensors' device as the current one: their
workspace and all of their launches belong to that device's current stream.  A stand-in
for a second device; CPU only."""
import contextlib

import torch

from w8a8_integer_linear_amd import _native as nat
from w8a8_integer_linear_amd import mlp


class Stop(Exception):
    pass


def test_passes_move_to_their_device(monkeypatch):
    at = []

    @contextlib.contextmanager
    def there(first, stream):
        assert stream is None
        at.append(first)
        try:
            yield
        finally:
            at.pop()

    def workspace(self, M):
        assert len(at) == 1
        raise Stop

    monkeypatch.setattr(nat, "_elsewhere", lambda first, stream: not at)
    monkeypatch.setattr(nat, "_there", there)
    monkeypatch.setattr(mlp.MLPW8A8Training, "_workspace", workspace)
    block = object.__new__(mlp.MLPW8A8Training)
    block.fc1 = block.fc2 = type("Layer", (), {"N": 64})()
    block.saved = dict(qx=torch.zeros((4, 32), dtype=torch.int8))
    x = torch.zeros((4, 32))
    for call in (block.forward, block.backward):
        try:
            call(x)
        except Stop:
            assert not at
        else:
            raise AssertionError("no workspace was asked for")
