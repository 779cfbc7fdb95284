"""Calls of the cache operators with a stream of the caller's: whose memory the outputs are made of, and how
long the inputs' stays theirs."""
import contextlib

import pytest
import torch

from long_context_prefill_rr_b200 import cache


class _Tensor:
    def __init__(self, made_on):
        self.made_on, self.used_on = made_on, []

    def record_stream(self, stream):
        self.used_on.append(stream)


@pytest.fixture
def fake(monkeypatch):
    """torch's streams and allocator with names in place of both: what is allocated belongs to the stream
    that is current then."""
    now = ["caller"]

    @contextlib.contextmanager
    def on(stream):
        now.append(stream)
        yield
        now.pop()

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[-1])
    monkeypatch.setattr(torch, "empty", lambda shape, dtype, device: _Tensor(now[-1]))


def test_outputs_are_allocated_for_the_stream_that_writes_them(fake):
    x = cache._new((4, 4), torch.bfloat16, "cuda:0", "side")
    assert x.made_on == "side" and x.used_on == ["caller"]
    x = cache._new((4, 4), torch.bfloat16, "cuda:0", None)
    assert x.made_on == "caller" and x.used_on == []


def test_tensors_of_a_call_are_kept_for_its_stream(fake):
    tensors = [_Tensor("caller"), None, _Tensor("caller")]
    cache._used("side", *tensors)
    assert tensors[0].used_on == tensors[2].used_on == ["side"]
    cache._used(None, *tensors)
    assert tensors[0].used_on == ["side"]


# ------------------------------------------------------------------------------------------ on the GPU
B, HQ, HKV, D, N = 3, 8, 2, 128, 64
CYCLES = 40_000_000       # 20 to 30 ms


def _ready():
    c = cache.PagedCache.allocate(B, 4 * N, HQ, HKV, D, page_size=16)
    g = torch.Generator(device="cuda").manual_seed(5)
    c.k.copy_(torch.randn(c.k.shape, generator=g, device="cuda"))
    c.v.copy_(torch.randn(c.v.shape, generator=g, device="cuda"))
    c.lengths.copy_(torch.tensor([N, 3, 17], dtype=torch.int32))
    x = torch.randn(B, HQ + 2 * HKV, N, D, generator=g, device="cuda").bfloat16()
    pos = torch.arange(N, dtype=torch.int32, device="cuda").expand(1, B, N).contiguous()
    torch.cuda.synchronize()
    return c, cache.RopeTable(D), pos, x[:, :HQ].clone(), x[:, HQ:HQ + HKV].clone(), x[:, HQ + HKV:].clone()


def _calls(c, table, pos, q, k, v, stream=None):
    """One call of each operator that makes outputs, as functions."""
    one = q[:, :, 0].contiguous()
    new = torch.full((B,), N, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    return {"decode": lambda: [c.decode(one, stream=stream)],
            "rope": lambda: list(cache.rope(table, pos, q, k, v, stream=stream)),
            "append": lambda: list(c.append(table, pos, q, k, v, new_len=new, k_out=True, v_out=True,
                                            advance=False, stream=stream))}


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["decode", "rope", "append"])
def test_outputs_do_not_take_memory_that_the_current_stream_still_writes(cuda_device, name):
    ready = _ready()
    ref = _calls(*ready)[name]()
    side = torch.cuda.Stream()
    call = _calls(*ready, stream=side)[name]
    torch.cuda.synchronize()
    # blocks of the outputs' sizes, freed while a slow kernel and a fill of them are still to run
    old = [torch.empty_like(x) for x in ref]
    torch.cuda._sleep(CYCLES)
    for x in old:
        x.fill_(7.0)
    where = {x.data_ptr() for x in old}
    del old, x
    got = call()
    side.synchronize()
    early = [x.clone() for x in got]
    torch.cuda.synchronize()
    assert not where & {x.data_ptr() for x in got}
    for a, b, c in zip(ref, early, got):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["decode", "rope", "append"])
def test_inputs_may_be_dropped_after_the_call(cuda_device, name):
    c, table, pos, q, k, v = _ready()
    ref = _calls(c, table, pos, q, k, v)[name]()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    sizes = [x.shape for x in (q, k, v)] + [q[:, :, 0].shape]
    one = q[:, :, 0].contiguous()
    new = torch.full((B,), N, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    where = {x.data_ptr() for x in (q, k, v, one, pos, new)}
    with torch.cuda.stream(side):
        torch.cuda._sleep(CYCLES)
    if name == "decode":
        got = [c.decode(one, stream=side)]
        where -= {x.data_ptr() for x in (q, k, v, pos, new)}
    elif name == "rope":
        got = list(cache.rope(table, pos, q, k, v, stream=side))
        where -= {one.data_ptr(), new.data_ptr()}
    else:
        got = list(c.append(table, pos, q, k, v, new_len=new, k_out=True, v_out=True, advance=False,
                            stream=side))
        where -= {one.data_ptr()}
    del q, k, v, one, pos, new
    late = [torch.full(s, 7.0, dtype=torch.bfloat16, device="cuda") for s in sizes]
    late += [torch.full((1, B, N), 7, dtype=torch.int32, device="cuda"),
             torch.full((B,), 1, dtype=torch.int32, device="cuda")]
    assert not where & {x.data_ptr() for x in late}
    torch.cuda.synchronize()
    for a, b in zip(ref, got):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_a_captured_call_on_a_stream_beside(cuda_device):
    """A capture that forks: the outputs come out of the graph's own memory, and replay after replay gives
    the same."""
    ready = _ready()
    ref = [x.clone() for name in ("append", "decode") for x in _calls(*ready)[name]()]
    side, got = torch.cuda.Stream(), []
    calls = _calls(*ready, stream=side)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        for name in ("append", "decode"):
            got += calls[name]()
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for x in got:
            x.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(ref, got):
            assert torch.equal(a, b)
