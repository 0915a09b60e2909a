"""Calls with an explicit stream that waits for nothing: what they allocate
must be no block that the current stream gave up and still reads, and their
results must not be handed out again while the current stream reads them."""
import pytest
import torch

from _parity import dev

pytestmark = pytest.mark.gpu

PAUSE = 40_000_000  # cycles that the current stream is kept busy: some 20 ms


def _route(moe, g):
    l = torch.randn((65536, 64), generator=g, device=dev())
    return lambda s: moe.moe_route_scored(l, 8, score=1, stream=s)


def _route_grad(moe, g):
    l = torch.randn((16384, 64), generator=g, device=dev())
    ids, w, _ = moe.moe_route_scored(l, 4)
    return lambda s: moe.moe_route_scored_backward(l, ids, w, z_coef=0.1, stream=s)


def _combine_grad(moe, g):
    T, k, H = 512, 4, 1024
    y = torch.randn((T * k, H), generator=g, device=dev())
    d_out = torch.randn((T, H), generator=g, device=dev()).bfloat16()
    inv = torch.randperm(T * k, generator=g, device=dev()).int()
    w = torch.rand((T, k), generator=g, device=dev())
    kd = torch.full((1,), k, dtype=torch.int32, device=dev())
    return lambda s: moe.moe_combine_backward(d_out, y, inv, w, kd, stream=s)


def _lora(T, n, R, K=1024, N=2048):
    def make(moe, g):
        x = torch.randn((T, K), generator=g, device=dev()).bfloat16()
        a = (torch.randn((n, R, K), generator=g, device=dev()) * K ** -0.5).bfloat16()
        b = torch.randn((n, N, R), generator=g, device=dev()).bfloat16()
        base = torch.randn((T, N), generator=g, device=dev())
        ids = torch.randint(-1, n, (T,), generator=g, device=dev(), dtype=torch.int32)
        return lambda s: (moe.moe_lora_apply(x, ids, a, b, None, base, stream=s),)
    return make


def _logits(moe, g):
    x = torch.randn((16384, 256), generator=g, device=dev()).bfloat16()
    w = torch.randn((64, 256), generator=g, device=dev())
    return lambda s: (moe.moe_router_logits(x, w, stream=s),)


def _permute(moe, g):
    ids = torch.randint(-1, 64, (65536, 8), generator=g, device=dev(), dtype=torch.int32)
    kd = torch.full((1,), 8, dtype=torch.int32, device=dev())
    return lambda s: moe.moe_permute_masked(ids, kd, 64, stream=s)


CALLS = dict(route=_route, route_grad=_route_grad, combine_grad=_combine_grad,
             lora_rows=_lora(64, 4, 8), lora_grouped=_lora(2048, 8, 32), logits=_logits,
             permute=_permute)


def make(moe, name):
    g = torch.Generator(device=dev())
    g.manual_seed(len(name))
    call = CALLS[name](moe, g)
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    return call, want


def same(a, b):
    return len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("name", CALLS)
def test_memory_of_the_current_stream_is_left_to_it(cuda_lib, name):
    """Blocks of the results' sizes are dropped while the current stream has
    yet to copy them; the call on the other stream runs at once."""
    call, want = make(cuda_lib, name)
    side = torch.cuda.Stream()
    sizes = [t.numel() * t.element_size() for t in want] * 2 + [1 << 12, 1 << 16, 1 << 20, 1 << 21]
    old = [torch.full((n,), 7, dtype=torch.uint8, device=dev()) for n in sizes]
    kept = [torch.zeros_like(o) for o in old]
    torch.cuda.synchronize()
    torch.cuda._sleep(PAUSE)
    for k, o in zip(kept, old):
        k.copy_(o)
    del o, old
    got = call(side)
    torch.cuda.synchronize()
    assert all((k == 7).all() for k in kept)
    assert same(got, want)


@pytest.mark.parametrize("name", CALLS)
def test_results_are_not_handed_out_while_they_are_read(cuda_lib, name):
    """The results of one call are copied late by the current stream and
    dropped; a second call on the same stream must not write over them."""
    call, want = make(cuda_lib, name)
    side = torch.cuda.Stream()
    kept = [torch.zeros_like(t) for t in want]
    torch.cuda.synchronize()
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(PAUSE)
    for k, t in zip(kept, got):
        k.copy_(t)
    sizes = [t.numel() * t.element_size() for t in got]
    del t, got
    with torch.cuda.stream(side):
        for n in sizes:
            torch.full((n,), 9, dtype=torch.uint8, device=dev())
    again = call(side)
    torch.cuda.synchronize()
    assert same(kept, want) and same(again, want)


def test_grouped_adapters_on_two_streams_without_workspaces(cuda_lib):
    """A grouped call on the current stream, whose workspace is dropped at
    once, and one of another shape on a second stream behind no wait."""
    first, want1 = make(cuda_lib, "lora_grouped")
    g = torch.Generator(device=dev())
    g.manual_seed(99)
    second = _lora(3000, 40, 16)(cuda_lib, g)
    want2 = [t.clone() for t in second(None)]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    cuda_lib.moe_get_device_error(clear=True)
    for _ in range(5):
        torch.cuda._sleep(PAUSE // 10)
        got1 = first(None)
        got2 = second(side)
        got3 = first(None)
        torch.cuda.synchronize()
        assert same(got1, want1) and same(got2, want2) and same(got3, want1)
    assert cuda_lib.moe_get_device_error(clear=True) == 0


def test_a_stream_given_as_the_default_one(cuda_lib):
    """stream=torch.cuda.default_stream() while another one is current."""
    call, want = make(cuda_lib, "route")
    with torch.cuda.stream(torch.cuda.Stream()):
        got = call(torch.cuda.default_stream())
    torch.cuda.synchronize()
    assert same(got, want)
