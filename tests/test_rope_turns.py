"""Frequencies that the rotation's table cannot hold."""
import math

import pytest
import torch

import sparse_attention_speculative_gb300 as vsd


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_frequencies_that_are_no_numbers(bad):
    for f in ([1.0, bad], torch.tensor([bad, 0.5]), torch.tensor([bad], dtype=torch.float64)):
        with pytest.raises(ValueError, match="finite"):
            vsd.vsd_rope_turns(f, device="cpu")


def test_no_frequency():
    t = vsd.vsd_rope_turns([], device="cpu")
    assert t.dtype == torch.int64 and t.shape == (0,)
