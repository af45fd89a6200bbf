"""8-bit caches without a GPU: tensors of a cache that change between calls, captures on a device that is not the current
one, and the frequencies of positions scaled for long contexts."""
import contextlib
import math

import pytest
import torch

import block_sparse_attention_06_gb300 as m


# ------------------------------------------------------------------------------------------------ caches

SWAPS = [("k", lambda x: torch.zeros(4)), ("k", lambda x: x[:2].clone()), ("v", lambda x: x[:2].clone()),
         ("kidx", lambda x: x[:, :, :, ::2].clone()), ("kidx", lambda x: x.transpose(0, 1)),
         ("v_scale", lambda x: x[:2].clone()), ("k_scale", lambda x: torch.zeros(x.shape)),
         ("kidx_scale", lambda x: x.view(torch.uint8))]


@pytest.mark.parametrize("name,swap", SWAPS)
def test_tensors_of_a_cache_are_looked_at_in_every_call(name, swap):
    """A tensor keeps its place in the cache while its storage changes (a pool made smaller, another type): refused in
    the next call, as by a cache made anew."""
    dims = m.Dims(16, 4, 128, 64, 4, 3)
    c = m.CacheQ8.zeros(dims, 8, "cpu")
    dev = c.k.get_device()               # of a tensor on the host: stands for any device here
    for _ in range(2):
        assert c._struct(dims, dev, True, True)[1] == 8
    x = getattr(c, name)
    x.data = swap(x)
    for cache in (c, m.CacheQ8(c.k, c.k_scale, c.v, c.v_scale, c.kidx, c.kidx_scale)):
        with pytest.raises((TypeError, ValueError)):
            cache._struct(dims, dev, True, True)


def test_a_cache_that_grows_is_taken_as_it_is():
    dims = m.Dims(16, 4, 128, 64, 4, 3)
    c, big = m.CacheQ8.zeros(dims, 2, "cpu"), m.CacheQ8.zeros(dims, 5, "cpu")
    dev = c.k.get_device()
    assert c._struct(dims, dev, True, False)[1] == 2
    for name in ("k", "k_scale", "v", "v_scale"):
        getattr(c, name).data = getattr(big, name)
    assert c._struct(dims, dev, True, False)[1] == 5


# ------------------------------------------------------------------------------------------------ captures

def test_a_step_is_captured_and_replayed_on_its_own_device(monkeypatch):
    """On a machine with several GPUs, of which another one is current: recorded stand-ins for torch's calls."""
    state = {"device": 0, "capture": None}
    seen = []

    @contextlib.contextmanager
    def device(d):
        old, state["device"] = state["device"], torch.device(d).index if not isinstance(d, int) else d
        yield
        state["device"] = old

    class Stream:
        def __init__(self, d=None):
            self.device = state["device"] if d is None else torch.device(d).index

    @contextlib.contextmanager
    def graph(g, pool=None, stream=None):
        old = dict(state)
        state["capture"] = 0 if stream is None else stream.device               # torch's own capture stream is the first device's
        state["device"] = state["capture"]
        yield
        state.update(old)

    class Graph:
        def replay(self):
            seen.append(("replay", state["device"]))

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "graph", graph)
    monkeypatch.setattr(torch.cuda, "CUDAGraph", Graph)
    monkeypatch.setattr(torch.cuda, "synchronize", lambda d=None: None)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state["device"], raising=False)

    class Q:
        device = torch.device("cuda", 1)
        is_cuda = True

        def get_device(self):
            return 1

    for cls, n in ((m.DecodeStepQ8, 9), (m.DecodeStep, 7)):
        step = cls.__new__(cls)
        step.out, step.lse, step._graph_results = "out", "lse", ("out", "lse")
        run = lambda *a, **k: seen.append(("step", state["capture"], state["device"]))  # noqa: E731
        monkeypatch.setattr(cls, "step" if cls is m.DecodeStepQ8 else "__call__",
                            (lambda f: lambda self, *a, **k: f(*a, **k))(run))
        seen.clear()
        step.capture(Q(), *[None] * (n - 1))
        assert seen[0][:2] == ("step", None) and seen[1] == ("step", 1, 1), cls
        assert state == {"device": 0, "capture": None}
        step.replay()
        assert seen[2] == ("replay", 1) and state["device"] == 0, cls


# ------------------------------------------------------------------------------------------------ frequencies

@pytest.mark.parametrize("rot,base,factor,length", [(64, 10000.0, 16.0, 4096), (128, 500000.0, 4.0, 8192), (32, 10000.0, 2.0, 512)])
def test_yarn_is_its_definition(rot, base, factor, length):
    """A pair that turns r times over the original length keeps its frequency for r above beta_fast, is divided by the
    factor below beta_slow, and is blended linearly in the pair's number between the two (their whole pairs outwards)."""
    got, gain = m.rope_inv_freq(rot, base, "yarn", factor, length)
    # pair i turns length * base^(-2 i / rot) / (2 pi) times: the first that turns at most r times
    def at(r):
        i = 0.0
        lo, hi = -1000.0, 1000.0
        for _ in range(200):
            i = (lo + hi) / 2
            lo, hi = (i, hi) if length * base ** (-2 * i / rot) / (2 * math.pi) > r else (lo, i)
        return i
    lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
    for i in range(rot // 2):
        f = base ** (-2 * i / rot)
        kept = 1.0 if i <= lo else 0.0 if i >= hi else (hi - i) / (hi - lo)
        assert math.isclose(float(got[i]), f * kept + f / factor * (1 - kept), rel_tol=1e-12), i
    assert 0 < lo + 1 < hi < rot and math.isclose(gain, 0.1 * math.log(factor) + 1)
