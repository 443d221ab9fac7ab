"""Rows of probabilities that share memory are refused by verify_drafts, with the stride that they have: a kernel that took
rows of vocab for granted would read past their end. Needs no GPU: validation fails before any HIP call."""
import pytest
import torch

from post_int4_weight_amd import api

VOCAB = 10


def _ints(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


@pytest.mark.parametrize("name", ["target", "draft"])
@pytest.mark.parametrize("stride", [0, 1, VOCAB - 1])
def test_rows_that_overlap(monkeypatch, name, stride):
    monkeypatch.setattr(api, "_on_gpu", lambda t, name: None)
    monkeypatch.setattr(api, "_stream", lambda t: None)
    rows = {n: torch.full((3, VOCAB), 0.1) for n in ("target", "draft")}
    rows[name] = torch.full((3 * VOCAB,), 0.1).as_strided((3, VOCAB), (stride, 1))
    with pytest.raises(api.PTQError, match=f"row stride {stride} of {name} < vocab = {VOCAB}"):
        api.verify_drafts(rows["target"], _ints(3), _ints(3), _ints(2), torch.zeros(3), torch.zeros(1), draft=rows["draft"])


def test_a_broadcast_row_is_refused(monkeypatch):
    monkeypatch.setattr(api, "_on_gpu", lambda t, name: None)
    one = torch.full((1, VOCAB), 0.1)
    assert api._probabilities(one.expand(3, VOCAB), 3, VOCAB, "target") == 0
    assert api._probabilities(torch.zeros(3, 16)[:, :VOCAB], 3, VOCAB, "target") == 16
    # a single row, or none, has no stride to go by
    assert api._probabilities(one.as_strided((1, VOCAB), (3, 1)), 1, VOCAB, "target") == VOCAB
    assert api._probabilities(torch.zeros(0, VOCAB), 0, VOCAB, "target") == VOCAB
