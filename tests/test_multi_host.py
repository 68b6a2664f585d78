"""The host side of MultiAdamW, StateCodec8 and the 8-bit engine without a GPU: the order of work between streams, what
is kept alive and for how long, and what is refused.  Streams, tensors and the library are stand-ins that write a log."""
import gc
import weakref

import pytest
import torch

from zero_partitioned_mixed_replica_gb300 import engine, multi


class Stream:
    def __init__(self, name, log):
        self.name, self.log = name, log

    def wait_stream(self, other):
        if other is not self:
            self.log.append("%s waits for %s" % (self.name, other.name))


class Tensor:
    """Whatever touches its elements does so on the current stream."""

    def __init__(self, log):
        self.log = log

    def copy_(self, other):
        self.log.append("write")

    def clone(self):
        self.log.append("read")
        return self

    device, dtype = torch.device("cuda", 0), torch.float32

    def numel(self):
        return 5

    def data_ptr(self):
        return 256

    def record_stream(self, stream):
        self.streams = getattr(self, "streams", []) + [stream]


def _wide(monkeypatch, own_stream):
    """A MultiAdamW with 32-bit states on a stream of its own or on the current one, and the log."""
    log = []
    cur = Stream("current", log)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: cur)
    monkeypatch.setattr(multi, "_check_list", lambda *a: None)
    opt = multi.MultiAdamW.__new__(multi.MultiAdamW)
    opt.device, opt.state_bits, opt.numels = torch.device("cuda", 0), 32, [5, 6]
    opt.stream = Stream("own", log) if own_stream else None
    opt.m, opt.v = [Tensor(log), Tensor(log)], [Tensor(log), Tensor(log)]
    return opt, log


def test_loading_waits_for_the_step_under_way_and_the_next_step_for_the_loading(monkeypatch):
    opt, log = _wide(monkeypatch, own_stream=True)
    opt.load_states([0, 0], [0, 0])
    assert log == ["current waits for own"] + 4 * ["write"] + ["own waits for current"]
    opt, log = _wide(monkeypatch, own_stream=False)
    opt.load_states([0, 0], [0, 0])
    assert log == 4 * ["write"]


def test_the_next_step_waits_for_states_that_are_read(monkeypatch):
    opt, log = _wide(monkeypatch, own_stream=True)
    opt.states32()
    assert log == ["current waits for own"] + 4 * ["read"] + ["own waits for current"]
    opt, log = _wide(monkeypatch, own_stream=False)
    opt.states32()
    assert log == 4 * ["read"]


def test_the_executor_never_gets_8_bit_states(monkeypatch):
    # it would read and write four bytes an element of them
    eng = engine.ZeroStep.__new__(engine.ZeroStep)
    eng.state_bits, eng._args, eng.hp, eng.transient_hook = 8, "arguments", None, None
    eng._args_hp = eng._args_hook = None
    with pytest.raises(ValueError, match="8-bit"):
        eng.step_args()
    eng.state_bits = 32
    assert eng.step_args() == "arguments"


class Library:
    """Calls succeed and note the device that is current."""

    def __init__(self, log, current):
        self.log, self.current = log, current

    def __getattr__(self, name):
        def call(*a):
            self.log.append((name, self.current[-1]))
            return 0
        return call


class List:
    """A bound list that only keeps what it was bound with."""

    def __init__(self, *a):
        self.M = type("Handle", (), {"handle": 1})
        self.workspace, self.info = Tensor([]), None

    def bind(self, stream, **arrays):
        self.arrays = arrays


def _stand_in(monkeypatch, library=None):
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream("current", []))
    monkeypatch.setattr(multi, "_current_device", lambda: Tensor.device.index)
    monkeypatch.setattr(multi, "_check_list", lambda *a: None)
    monkeypatch.setattr(multi, "BoundList", List)
    monkeypatch.setattr(multi.B, "lib", lambda: library or Library([], [0]))


def _codec(monkeypatch, stream, library=None):
    _stand_in(monkeypatch, library)
    return multi.StateCodec8(*[[Tensor([]), Tensor([])] for _ in range(6)], stream)


def test_memory_in_use_on_another_stream_is_not_given_away_with_the_last_reference(monkeypatch):
    own = Stream("own", [])
    for stream in (own, None):
        codec = _codec(monkeypatch, stream)
        used = [codec._list.workspace] + [x for xs in codec._list.arrays.values() for x in xs]
        assert len(used) == 13
        assert all(getattr(x, "streams", []) == ([own] if stream else []) for x in used)
        opt, _ = _wide(monkeypatch, own_stream=False)
        opt.stream, opt.master, opt.out16, opt._list, opt.grads, opt._index = stream, None, None, List(), [Tensor([])], 0
        opt.rebind_grads([Tensor([]), Tensor([])])
        assert all(getattr(x, "streams", []) == ([own] if stream else []) for x in opt._list.arrays["grads"])


def _adamw(monkeypatch, library=None, **kw):
    _stand_in(monkeypatch, library)
    monkeypatch.setattr(multi, "_slices", lambda numels, dtype, device: [Tensor([]) for _ in numels])
    monkeypatch.setattr(multi.B, "zero_state_init", lambda *a: None)
    monkeypatch.setattr(torch, "zeros", lambda *a, **k: Tensor([]))
    return multi.MultiAdamW([Tensor([])], [Tensor([])], **kw)


def test_objects_go_with_their_last_reference(monkeypatch):
    # and their states' memory with them, not at some later collection of cycles
    gc.disable()
    try:
        for make in (lambda: _codec(monkeypatch, None), lambda: _adamw(monkeypatch), lambda: _adamw(monkeypatch, state_bits=8)):
            obj = make()
            gone = weakref.ref(obj)
            del obj
            assert gone() is None
    finally:
        gc.enable()


def test_calls_go_to_the_device_of_the_tensors(monkeypatch):
    """With another device current, a launch would go there with this one's addresses."""
    current, log = [0], []

    class On:
        def __init__(self, device):
            self.index = torch.device(device).index if not isinstance(device, int) else device

        def __enter__(self):
            current.append(self.index)

        def __exit__(self, *a):
            current.pop()

    library = Library(log, current)
    monkeypatch.setattr(torch.cuda, "device", On)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[-1])
    monkeypatch.setattr(Tensor, "device", torch.device("cuda", 1))
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    opts = [_adamw(monkeypatch, library, decide=True), _adamw(monkeypatch, library, state_bits=8)]
    codec = _codec(monkeypatch, None, library)
    monkeypatch.setattr(multi, "_current_device", lambda: current[-1])
    monkeypatch.setattr(multi, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(List, "bind", lambda self, stream, **arrays: log.append(("bind", current[-1])))
    monkeypatch.setattr(multi.B, "zero_state_init", lambda *a: log.append(("init", current[-1])))
    for opt in opts:
        opt.step()
    codec.encode()
    codec.decode()
    opts[0].rebind_grads([Tensor([])])
    assert [n for n, _ in log] == ["zero_multi_grad_norm", "zero_multi_adamw", "zero_multi_adamw8", "zero_multi_encode8",
                                   "zero_multi_decode8", "bind"]
    assert {d for _, d in log} == {1} and current == [0]


class Shards(Tensor):
    """[N_d, S] on the current stream."""

    shape = (1, 5)

    def to(self, *a, **k):
        return self

    def view(self, *a):
        return self

    def zero_(self):
        self.log.append("write")

    def __getitem__(self, at):
        return self


@pytest.mark.parametrize("own_stream", [True, False])
def test_the_engine_s_loads_and_reads_are_ordered_with_its_steps(monkeypatch, own_stream):
    log = []
    cur = Stream("current", log)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: cur)
    monkeypatch.setattr(torch, "zeros", lambda *a, **k: Shards(log))
    eng = engine.ZeroStep.__new__(engine.ZeroStep)
    eng.device, eng.stream, eng.state_bits, eng.n_d = torch.device("cuda", 0), Stream("own", log) if own_stream else None, 32, 1
    eng.info = type("Info", (), {"psi_pad": 5})
    eng.units = [type("Unit", (), {"offset": 0, "shard": 5, "shard_base": 0})]
    eng.master, eng.m, eng.v = Shards(log), Shards(log), Shards(log)
    eng.shard16 = eng.params = eng.gshard = None
    waits = ["current waits for own", "own waits for current"] if own_stream else []
    eng.load_master(Shards(log))
    assert log == waits[:1] + 3 * ["write"] + waits[1:]
    log.clear()
    eng.flat("master")
    assert log == waits[:1] + ["write"] + waits[1:]
