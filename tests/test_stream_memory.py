"""What the binding allocates for a call on a stream other than the current one is taken
in that stream's order (no GPU needed: the tensors claim to be on one, the library's
functions and the current stream are stand-ins)."""
import contextlib
import types

import pytest

torch = pytest.importorskip("torch")


class OnDevice(torch.Tensor):
    """A CPU tensor that says it is on cuda:0 and notes what is allocated from it."""
    taken = {}                 # address -> the stream current at its allocation
    held = {}                  # address -> streams recorded
    current = None
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0

    @classmethod
    def __torch_function__(cls, func, types, args=(), kwargs=None):
        t = super().__torch_function__(func, types, args, kwargs or {})
        if func in (torch.empty_like, torch.Tensor.new_empty) and t.numel():
            cls.taken[t.data_ptr()] = (cls.current, t)                 # (kept alive)
        return t

    def record_stream(self, stream):
        OnDevice.held.setdefault(self.data_ptr(), []).append(stream)


def tensor(*shape, dtype=torch.float16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)


def stream(name):
    return types.SimpleNamespace(name=name, cuda_stream=0, device=types.SimpleNamespace(index=0))


@pytest.fixture
def env(monkeypatch):
    import weight_only_quantization_b200 as hqq
    main, side = stream("main"), stream("side")
    OnDevice.taken, OnDevice.held, OnDevice.current = {}, {}, main

    @contextlib.contextmanager
    def entered(s):
        before, OnDevice.current = OnDevice.current, s
        yield
        OnDevice.current = before
    monkeypatch.setattr(torch.cuda, "stream", entered)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: OnDevice.current)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    calls = []

    class Lib:
        def __getattr__(self, name):
            if name.endswith(("_bytes", "_groups")):
                return getattr(real, name)
            return lambda *args: calls.append(args) or 0
    real = hqq._lib
    monkeypatch.setattr(hqq, "_lib", Lib())
    return types.SimpleNamespace(hqq=hqq, main=main, side=side, calls=calls)


def matrix(hqq):
    return hqq.QuantizedMatrix(tensor(64 * 128 // 2, dtype=torch.uint8), tensor(64, 2),
                               tensor(64, 2), 64, 128, 4, 64)


def check(env, results, passed=1):
    """Every allocation was the side stream's; results are held for the main one, what
    stayed inside the call needs no hold; all of them reached the library."""
    assert OnDevice.taken and len(env.calls) == passed
    mine = {r.data_ptr() for r in results}
    for at, (s, _) in OnDevice.taken.items():
        assert s is env.side
        assert at in [a for c in env.calls for a in c]
        assert OnDevice.held.get(at, []) == ([env.main] if at in mine else [])
    assert mine <= set(OnDevice.taken)
    assert OnDevice.current is env.main


def test_adapter_calls(env):
    q = matrix(env.hqq)
    ad = env.hqq.Adapters(tensor(2, 8, 128), tensor(2, 64, 8))
    index = tensor(3, dtype=torch.int32)
    X, dY = tensor(3, 128), tensor(3, 64)
    out = env.hqq.hqq_linear_adapters(X, q, ad, index, stream=env.side)
    check(env, [out])
    assert len(OnDevice.taken) == 2                      # the result and a workspace
    OnDevice.taken, OnDevice.held = {}, {}
    env.calls.clear()
    check(env, env.hqq.hqq_linear_adapters_backward(dY, X, q, ad, index, stream=env.side))
    assert len(OnDevice.taken) == 4


def test_distill(env):
    z, top, at = tensor(4, 100), tensor(4, 5), tensor(4, 5, dtype=torch.int64)
    check(env, env.hqq.hqq_distill(z, top, at, grad=True, stream=env.side))


# (results stay with the caller; what torch.empty makes is seen when it is held)
CALLS = {
    "quantize": lambda h, s: h.hqq_quantize(tensor(64, 128), stream=s),
    "quantize_ex": lambda h, s: h.hqq_quantize_ex(tensor(64, 128), stream=s),
    "quantize_half": lambda h, s: h.hqq_quantize_ex(tensor(64, 128), stream=s, precision="fp16"),
    "dequantize": lambda h, s: h.hqq_dequantize(matrix(h), stream=s),
    "meta_quantize": lambda h, s: h.hqq_meta_quantize(tensor(128), 16, stream=s),
    "meta_batch": lambda h, s: h.hqq_meta_quantize_batch([(tensor(128), 0), (tensor(64), 16)],
                                                         stream=s),
    "meta_dequantize": lambda h, s: h.hqq_meta_dequantize(meta(), stream=s),
    "dequantize_meta": lambda h, s: h.hqq_dequantize_meta(
        tensor(64 * 64, dtype=torch.uint8), meta(), 64, 128, 4, 64, scale=tensor(64, 2), stream=s),
    "linear": lambda h, s: h.hqq_linear(tensor(3, 128), matrix(h), stream=s),
    "linear_meta": lambda h, s: h.hqq_linear_meta(
        tensor(3, 128), tensor(64 * 64, dtype=torch.uint8), meta(), 64, 128, 4, 64,
        scale=tensor(64, 2), stream=s),
    "lowrank": lambda h, s: h.hqq_lowrank(tensor(64, 128), matrix(h), 8,
                                          tensor(128, 16, dtype=torch.float32), stream=s),
}


def flat(result):
    if isinstance(result, torch.Tensor):
        yield result
    elif result is not None and not isinstance(result, (int, float)):
        for r in result if isinstance(result, (tuple, list)) else vars(result).values():
            yield from flat(r)


def meta():
    import weight_only_quantization_b200 as hqq
    return hqq.Meta8(tensor(128, dtype=torch.uint8), tensor(1), tensor(1), 0)


@pytest.mark.parametrize("name", list(CALLS))
def test_earlier_calls(env, name, monkeypatch):
    """The library is called with the side stream current, all that the call made was
    made then, and its results are held for the main stream."""
    made = {}

    def empty(*args, device=None, **kwargs):
        t = real(*args, **kwargs).as_subclass(OnDevice)
        made[t.data_ptr()] = (OnDevice.current, t)
        return t
    real = torch.empty
    monkeypatch.setattr(torch, "empty", empty)
    result = CALLS[name](env.hqq, env.side)
    results = list(flat(result))
    assert made and results and len(env.calls) == 1
    mine = {t.data_ptr() for t in results}
    for at, (s, _) in made.items():
        assert s is env.side
        assert OnDevice.held.get(at, []) == ([env.main] if at in mine else [])
    assert mine <= set(made) and OnDevice.current is env.main
    assert len(made) == len(mine) + (name == "lowrank")          # its workspace


def test_the_current_stream_given_is_no_other_stream(env):
    z, top, at = tensor(4, 100), tensor(4, 5), tensor(4, 5, dtype=torch.int64)
    env.hqq.hqq_distill(z, top, at, grad=True, stream=env.main)
    env.hqq.hqq_distill(z, top, at, grad=True)
    assert not OnDevice.held and all(s is env.main for s, _ in OnDevice.taken.values())
