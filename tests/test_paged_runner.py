"""CPU tests of PagedRunner's streams: which stream a call's workspace and a plan's
memory are tied to, with stand-ins for CUDA's streams and for the library's calls."""
import threading
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")

from chunked_prefill_mixed_gb300 import runner as M  # noqa: E402


class Memory:
    """Device memory (a packed plan, a table): the streams that it was recorded for."""

    def __init__(self):
        self.recorded = []

    def record_stream(self, stream):
        self.recorded.append(stream.cuda_stream)


def _stream(raw):
    return SimpleNamespace(cuda_stream=raw, synchronize=lambda: None)


class Cuda:
    """Streams by their handles, all of device 0; what is made under which of them."""

    def __init__(self, monkeypatch):
        self.current, self.device, self.captured, self.zeroed = 0, 0, set(), []
        self.at = monkeypatch.setattr
        self.at(torch._C, "_cuda_getCurrentRawStream", lambda device: self.current, raising=False)
        self.at(torch.cuda, "is_current_stream_capturing", lambda: self.device == 0 and self.current in self.captured)
        self.at(torch._C, "_cuda_getDevice", lambda: self.device, raising=False)
        # (ExternalStream makes a stream of its own of the handle 0, as torch's does)
        self.at(torch.cuda, "ExternalStream", lambda raw, device=None: _stream(raw or 0x999))
        self.at(torch.cuda, "default_stream", lambda device=None: _stream(0))
        self.at(torch.cuda, "current_stream", lambda device=None: _stream(self.current))
        self.at(torch.cuda, "stream", self.under)
        self.at(torch, "zeros", self.zeros)

    def under(self, stream):
        cuda = self

        class Under:
            def __enter__(self):
                self.was = cuda.device, cuda.current
                cuda.device, cuda.current = 0, stream.cuda_stream

            def __exit__(self, *what):
                cuda.device, cuda.current = self.was
        return Under()

    def zeros(self, n, dtype=None, device=None):
        self.zeroed.append(self.current)
        return torch.empty(n, dtype=dtype).fill_(0)


@pytest.fixture
def made(monkeypatch):
    """A runner whose first stream is ``home``, the stand-ins and the library's calls."""
    calls = []

    def make(home):
        r = object.__new__(M.PagedRunner)
        r.device, r._home, r._retired, r._others = torch.device("cuda", 0), home, [], {}
        r._lock, r.workspace, r.rope, r.shape = threading.Lock(), torch.empty(1 << 16, dtype=torch.uint8), Memory(), None
        r.dtype = None
        r._calls, r._append = SimpleNamespace(attend="attend", append="append"), None
        monkeypatch.setattr(M, "_made", lambda call, *a: calls.append((call, a)))
        return r, Cuda(monkeypatch), calls
    return make


def _plan(home, nbytes=1 << 12):
    p = object.__new__(M.PagedPlan)
    p.info, p.dev, p.args, p.home, p.tokens, p.workspace_bytes = None, Memory(), None, home, 3, nbytes
    return p


@pytest.mark.parametrize("call_on", [0, 0x30])
@pytest.mark.parametrize("current", [0, 0x30, 0x70])
def test_a_workspace_is_zeroed_on_the_stream_of_its_calls(made, call_on, current):
    """Zeros are enqueued before the calls that need them, on the calls' own stream: the
    default one (handle 0) too, where the runner's first stream is another."""
    r, cuda, calls = made(0x10)
    cuda.current = current
    for nbytes in (1 << 12, 1 << 20):
        r.attend(_plan(call_on, nbytes), None, None, None, None, stream=call_on)
        assert cuda.zeroed[-1] == call_on and calls[-1][1][-1] == call_on
    r.append(None, None, None, None, None, None, stream=call_on)
    assert len(cuda.zeroed) == 2 and calls[-1][0] == "append" and calls[-1][1][-1] == call_on
    cuda.captured = {call_on}
    r.attend(_plan(call_on, 1 << 12), None, None, None, None, stream=call_on)
    assert calls[-1][1][4] is r.workspace and r._others[call_on] is not r.workspace


@pytest.mark.parametrize("home,plan_on,call_on,captured,recorded", [
    (0x10, 0x10, 0x10, False, False),   # made and used on the runner's first stream
    (0x10, 0x20, 0x10, False, True),    # made on another, used on the first
    (0x10, 0x10, 0x20, False, True),    # the other way round
    (0x10, 0x20, 0x20, False, False),   # made and used on another
    (0x10, 0x20, 0x30, False, True),
    (0x10, 0x20, 0x10, True, False),    # captured: the caller keeps the plan
    (0x10, 0x10, 0x20, True, False),
])
def test_a_plan_outlives_its_calls_on_other_streams(made, home, plan_on, call_on, captured, recorded):
    """The memory of a plan is not reused before a call on another stream than the plan's
    is done, whichever of the two is the runner's first."""
    for given in (True, False):      # the call's stream as an argument, or the current one
        r, cuda, calls = made(home)
        plan = _plan(plan_on)
        cuda.captured = {call_on} if captured else set()
        cuda.current = 0x70 if given else call_on
        r.attend(plan, None, None, None, None, stream=call_on if given else None)
        assert plan.dev.recorded == ([call_on] if recorded else [])
        assert calls[-1][0] == "attend" and calls[-1][1][-1] == call_on


@pytest.mark.parametrize("home", [0, 0x10])
@pytest.mark.parametrize("current", [0, 0x10, 0x20])
def test_the_runners_own_memory_outlives_its_calls(made, home, current):
    """A runner may be dropped while its last calls run: the main workspace is of the
    first stream's memory wherever a batch is planned, and the table is recorded once
    for every other stream that a call runs on."""
    r, cuda, calls = made(home)
    cuda.current = current
    assert not bool(r._zeros(256).any()) and cuda.zeroed == [home] and cuda.current == current
    for call_on in (0, 0x10, 0x20, 0x10, 0):
        r.append(None, None, None, None, None, None, stream=call_on)
        r.attend(_plan(call_on, 1 << 20), None, None, None, None, stream=call_on)
    assert r.rope.recorded == [s for s in (0, 0x10, 0x20) if s != home]
    r.rope = None                    # (a runner without a table)
    r.attend(_plan(0x40), None, None, None, None, stream=0x40)
    assert 0x40 in r._others


@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("call_on", [0, 0x20])
def test_a_capture_is_seen_from_another_device(made, call_on, given):
    """Whether a call is captured is asked of the runner's device, not of the current one."""
    r, cuda, calls = made(0x10)
    cuda.device, cuda.current, cuda.captured = 1, call_on, {call_on}
    r.attend(_plan(0x10), None, None, None, None, stream=call_on if given else None)
    assert calls[-1][1][4] is r.workspace and not r._others and cuda.device == 1


def test_tensors_of_another_type_than_the_runners_are_refused(made):
    """A runner for one element type takes that one (the other tensors have to be of the
    same as the first anyway); a runner for none takes both."""
    r, cuda, calls = made(0x10)
    cuda.current = 0x10
    bf, half = (torch.zeros(1, dtype=t) for t in (torch.bfloat16, torch.float16))

    def both(t):
        r.append(t, t, None, None, None, None)
        r.attend(_plan(0x10), t, None, None, None)
    both(bf), both(half)
    for mine, other in ((bf, half), (half, bf)):
        r.dtype = mine.dtype
        both(mine)
        n = len(calls)
        with pytest.raises(ValueError, match="k: .*the runner is for"):
            r.append(other, other, None, None, None, None)
        with pytest.raises(ValueError, match="q: .*the runner is for"):
            r.attend(_plan(0x10), other, None, None, None)
        assert len(calls) == n
