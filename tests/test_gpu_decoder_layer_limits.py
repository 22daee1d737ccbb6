"""The decoder layer example at the lengths it was made for, and past them."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_decoder_layer import ex, tokens  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def test_lengths_past_the_block_are_refused(ex):  # noqa: F811
    """More tokens than a sequence has room for would be written outside its pages and not be seen: refused before
    anything changes, and the block goes on as if the call had not been."""
    block, twin = (ex.random_block(256, 4, 2, 2, 70, 64) for _ in range(2))
    x, r = tokens(64, 256, 1)
    with pytest.raises(ValueError):
        block.load_prefix(*tokens(65, 256, 1))
    x2, r2 = tokens(69, 256, 2)
    for b in (block, twin):
        b.load_prefix(x, r)
        b.step(x2, r2, [68, 1])
    for counts in ([3, 0], [0, 70], [1], [-1, 4], [2, 0]):
        with pytest.raises(ValueError):
            block.step(*tokens(3, 256, 3), counts)
    x3, r3 = tokens(3, 256, 4)
    a, b = block.step(x3, r3, [2, 1]), twin.step(x3, r3, [2, 1])
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert block.own_len.tolist() == [70, 2]
