"""Beam selection of batches that shrink, on one workspace."""
import numpy as np
import pytest
import torch

from eagle_speculative_decoding_step_gb300 import binding as lib
from oracle import decode as oracle

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("W,V,most", [(4, 128256, 38), (8, 40000, 19), (1, 20000, 200)])
def test_a_workspace_of_the_largest_batch_serves_all_smaller_ones(W, V, most):
    g = torch.Generator(device="cuda").manual_seed(W)
    logits = torch.randn(most, W, V, generator=g, device="cuda") * 3
    score = -torch.arange(1, most * W + 1, device="cuda").float().view(most, W) / 7
    done = torch.zeros(most, W, dtype=torch.int32, device="cuda")
    ref = oracle.beam_select(logits.double().cpu().numpy(), score.cpu().numpy(), done.cpu().numpy(), 2)
    size = lib.spec_beam_workspace_bytes(most, W, V)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for B in sorted({most, most - 1, most // 2, 5, 3, 2, 1}, reverse=True):
        p, t, d = (torch.full((B, W), -7, dtype=torch.int32, device="cuda") for _ in range(3))
        s = torch.empty(B, W, device="cuda")
        lib.spec_beam_select(B, W, V, "f32", logits, score, done, 2, p, t, s, d, ws)
        assert lib.spec_get_device_error(ws) == 0
        np.testing.assert_array_equal(p.cpu().numpy(), ref[0][:B])
        np.testing.assert_array_equal(t.cpu().numpy(), ref[1][:B])
