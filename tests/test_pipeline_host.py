"""The order of FwdBwdPipeline's work, on fake streams that keep what each of them is ordered behind."""
import contextlib
import types

import pytest
import torch

import attention_attn_fwd_10_b200 as attn


class Event:
    def __init__(self):
        self.behind = frozenset()

    def record(self, stream):
        self.behind = frozenset(stream.behind)


class Stream:
    """`behind`: the work that whatever is enqueued next runs after."""

    def __init__(self, device=None):
        self.device, self.behind = device, set()

    def wait_event(self, event):
        self.behind |= event.behind

    def wait_stream(self, other):
        self.behind |= other.behind

    def synchronize(self):
        pass


class Frequencies:
    """Stands for a Rotary whose tensors the caller's stream writes."""

    def _struct(self, positions, tokens, dev):
        pass


@pytest.fixture
def fake(monkeypatch):
    caller = Stream()
    seen = []
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "Event", Event)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: caller)
    monkeypatch.setattr(attn, "bwd_workspace_size", lambda *a: 16)

    def kernel(name):
        def run(*a, stream=None, **kw):
            seen.append((name, set(stream.behind)))
            stream.behind.add(name)

        return run

    for name in ("rope", "fwd", "bwd"):
        monkeypatch.setattr(attn, name, kernel(name))
    return types.SimpleNamespace(caller=caller, seen=seen)


def _step(pipe):
    x = [torch.zeros((1, 4, 1, 64), dtype=torch.bfloat16) for _ in range(4)]
    out = {n: torch.zeros((1, 4, 1, 64), dtype=torch.bfloat16) for n in ("o", "dq", "dk", "dv")}
    pipe.submit(*x, out | {"lse": torch.zeros((1, 1, 4))})


def test_rotations_run_behind_the_caller_s_work(fake):
    positions = torch.zeros((1, 4), dtype=torch.int32)
    pipe = attn.FwdBwdPipeline(1, 4, 4, 1, 1, 64, device="cpu", rotary=Frequencies(), positions=positions)
    for step in ("positions of step 1", "positions of step 2"):  # the first written, then changed in place
        fake.caller.behind.add(step)
        fake.seen.clear()
        _step(pipe)
        assert [name for name, _ in fake.seen] == ["rope", "fwd", "bwd", "rope"]
        for name, behind in fake.seen:
            assert step in behind, f"{name} may run before the positions are written"


def test_without_rotation_the_steps_wait_for_nothing_of_the_caller(fake):
    pipe = attn.FwdBwdPipeline(1, 4, 4, 1, 1, 64, device="cpu")
    fake.caller.behind.add("something else")
    _step(pipe)
    assert [name for name, _ in fake.seen] == ["fwd", "bwd"]
    assert all("something else" not in behind for _, behind in fake.seen)


def test_positions_without_rotary_are_refused(fake):
    positions = torch.zeros((1, 4), dtype=torch.int32)
    with pytest.raises(ValueError, match="without rotary"):
        attn.FwdBwdPipeline(1, 4, 4, 1, 1, 64, device="cpu", positions=positions)
    x = torch.zeros((1, 4, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="without rotary"):
        attn.fwd_bwd(x, x, x, x, positions=positions)
