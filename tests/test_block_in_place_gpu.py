"""The layer and its block where the input is the memory of the result: the layer's
own reused buffer given back to it, or out=x."""
import pytest
import torch

from _parity import dev
from test_block_gpu import m, make, rand

pytestmark = pytest.mark.gpu


def test_shared_expert_reads_the_input_before_the_result_is_written():
    for T in (1, 7, 300):
        layer, _ = make(T=T)
        x = rand((T, 256), 7, 0.5)
        apart = [torch.empty_like(x), torch.empty_like(x)]
        layer(x, out=apart[0])
        layer(apart[0], out=apart[1])
        y = layer(x)
        assert torch.equal(y, apart[0])
        again = layer(y)  # the buffer that the call before returned
        assert again.data_ptr() == y.data_ptr() and torch.equal(again, apart[1])
        both = x.clone()
        assert layer(both, out=both) is both and torch.equal(both, apart[0])


def test_blocks_without_norms_take_the_buffer_of_their_result():
    layer, _ = make(out_norm=False)
    layer.norm = None
    x = rand((48, 256), 7, 0.5)
    first = layer.block(x)[0].clone()
    second = layer.block(first, out=torch.empty_like(x))[0]
    y, _ = layer.block(x)
    assert torch.equal(layer.block(y)[0], second)


def test_gradients_need_an_input_apart_from_the_result():
    layer, x = make(out_norm=False)
    layer.keep_for_grad = True
    d = rand(x.shape, 3, 0.1)
    y = layer(x)
    want = {n: t.clone() for n, t in layer.grads(d)[0].items()}
    for call in (lambda: layer(y), lambda: layer(x, out=x), lambda: layer(x[1:], out=x[:-1])):
        with pytest.raises(ValueError):  # grads() would read the result in the input's place
            call()
        with pytest.raises(ValueError):
            layer.grads(d)
    layer(x)
    assert all(torch.equal(t, want[n]) for n, t in layer.grads(d)[0].items())
    layer.keep_for_grad = False
    layer(x, out=x)  # nothing reads it again


def test_the_sum_of_a_block_is_not_its_result():
    for kw in (dict(), dict(out_norm=False)):
        layer, x = make(**kw)
        first, s = layer.block(x)
        assert s is x
        first = first.clone()
        second = layer.block(first)[0].clone()
        both = x.clone()
        y, s = layer.block(both, out=both)
        assert y is both and torch.equal(y, first) and torch.equal(s, x)
        y, _ = layer.block(x)
        y, s = layer.block(y)  # its own buffer once more
        assert torch.equal(y, second) and torch.equal(s, first)
        third, total = layer.block(x, residual=first)
        third, total = third.clone(), total.clone()
        _, mine = layer.block(x, residual=first)
        with pytest.raises(ValueError):
            layer.block(x, residual=first, out=mine)
        other = torch.empty_like(x)
        y, mine = layer.block(x, residual=first, out=other)
        assert torch.equal(y, third) and torch.equal(mine, total)
        # the sum may take the place of the one before
        y, again = layer.block(x, residual=mine)
        assert again.data_ptr() == mine.data_ptr()
        assert torch.equal(again, (x.float() + total.float()).to(torch.bfloat16))


def test_the_result_of_a_block_is_not_written_over_what_its_gradients_read():
    layer, x = make()
    d = rand(x.shape, 3, 0.1)
    y = layer(x)  # the rows that block() keeps for out_norm's gradient are this buffer
    layer.keep_for_grad = True
    layer.block(x)
    want = {n: t.clone() for n, t in layer.grads(d)[0].items()}
    with pytest.raises(ValueError):
        layer.block(x, out=y)
    same = x.clone()
    layer.block(same, out=same)  # the norm in front keeps rows of its own
    assert all(torch.equal(t, want[n]) for n, t in layer.grads(d)[0].items())
    layer.norm = None
    with pytest.raises(ValueError):
        layer.block(same, out=same)
    result, _ = layer.block(x)
    with pytest.raises(ValueError):
        layer.block(result)
    layer.keep_for_grad = False
    layer.block(x, out=y)
    layer.block(result)


def test_gradients_belong_to_the_parts_of_their_forward():
    """A shared expert or a norm that came, went or changed after the forward left no rows for
    its gradient."""
    layer, x = make()
    layer.keep_for_grad = True
    d = rand(x.shape, 3, 0.1)
    layer.block(x)
    want = {n: t.clone() for n, t in layer.grads(d)[0].items()}
    shared, norm = layer.shared, layer.out_norm
    moe = m()
    others = [("shared", None), ("shared", moe.SharedExpert(shared.gate_up.clone(), shared.down)),
              ("shared", moe.SharedExpert(rand((64, 256), 1), rand((256, 32), 2))), ("out_norm", None),
              ("out_norm", moe.Norm(norm.weight.clone(), norm.bias, norm.kind)),
              ("out_norm", moe.Norm(norm.weight, norm.bias, moe.NORM_RMS)),
              ("scoring", moe.ScoredRouting(score=moe.SCORE_SOFTMAX, n_groups=4, topk_groups=2, scale=2.0)),
              ("scoring", None)]
    scoring = layer.scoring
    for name, other in others:
        setattr(layer, name, other)
        with pytest.raises(ValueError):
            layer.grads(d)
        layer.shared, layer.out_norm, layer.scoring = shared, norm, scoring
    layer.out_norm = moe.Norm(norm.weight, norm.bias, norm.kind, float(str(norm.eps)))  # equal
    layer.scoring = moe.ScoredRouting(scoring.score, torch.zeros(layer.E, device=dev()), 4, 2, 2, 2.0)  # of the next call
    assert all(torch.equal(t, want[n]) for n, t in layer.grads(d)[0].items())
    layer.shared = None
    layer.block(x)
    layer.grads(d)
    layer.shared = shared  # no forward has passed it
    with pytest.raises(ValueError):
        layer.grads(d)
    layer(x)  # a forward alone leaves the norm out
    layer.out_norm = None
    assert "shared.down" in layer.grads(d)[0]


def test_the_sum_of_a_block_is_kept_from_every_buffer_that_the_block_writes():
    """A block's input may be what the layer alone returned before, in the buffer that stands
    between the layer and the norm behind it."""
    for norm in (True, False):
        layer, x = make()
        if not norm:
            layer.norm = None
        y = layer(x)
        first = y.clone()
        want = layer.block(first, out=torch.empty_like(x))[0]
        y = layer(x)
        got, s = layer.block(y)
        assert torch.equal(got, want) and torch.equal(s, first)
        normed = layer.buffers(x.shape[0]).get("normed")
        if normed is not None:
            normed.copy_(first)
            got, s = layer.block(normed)
            assert torch.equal(got, want) and torch.equal(s, first)
            layer.keep_for_grad = True
            with pytest.raises(ValueError):  # grads() reads the normed rows
                layer.block(first, out=normed)
