"""GPU cases at the edges of the calls for prompts and samples, against the fp64 oracle (tolerances: test_gpu_prompts)."""
import numpy as np
import pytest
import torch

from test_gpu_prompts import TYPE_PAIRS, TYPES, Chunk, error

pytestmark = pytest.mark.gpu


def far_below_zero(x, at=225.0):
    """Every score of x near -at: q = -a (1, 1, ...) + noise, k = 4 (1, 1, ...) + noise, 4 a sqrt(hd) = at."""
    g = torch.Generator(device="cuda").manual_seed(17)
    a = at / (4 * x.hd ** 0.5)
    x.wide.copy_(0.5 * torch.randn(x.wide.shape, generator=g, device="cuda") - a)
    same = torch.uint8 if x.c == "e4m3" else x.k.dtype
    k = ((4 + 0.5 * torch.randn(x.k.shape, generator=g, device="cuda")) / x.ks).to(TYPES[x.c])
    x.k.view(same).copy_(k.view(same))


@pytest.mark.parametrize("t,c", TYPE_PAIRS)
@pytest.mark.parametrize("hd", [64, 256])
@pytest.mark.parametrize("chunks,window", [([(40, 300), (3, 3)], 0),              # whole items
                                           ([(1, 5000)], 0), ([(3, 4100), (1, 2)], 0),     # pieces of one row's keys
                                           ([(150, 420), (1, 300)], 70),          # rows that see nothing of an item's first tile
                                           ([(200, 1900)], 700)])                 # or of a piece
def test_chunk_attention_scores_far_below_zero(t, c, hd, chunks, window):
    """The first scores that a row sees are no reference of 0: 2^(0 - s) would overflow."""
    x = Chunk(chunks, 4, 2, hd, t, c, window=window, seed=21)
    far_below_zero(x)
    out, lse, ws = x.run()
    assert error(ws) == 0
    x.check(out, lse)
    assert (lse[:int(x.cu[-1])] < -150).all()
