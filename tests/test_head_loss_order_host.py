"""The order of a LossHead's calls, on the CPU: backward() goes by what the last score()
left in the head's buffers, so it refuses another one's sums."""
import pytest
import torch

from checkpoint_averaging_amd import dlhead as dh
from checkpoint_averaging_amd import dlmerge as dl
from checkpoint_averaging_amd.head import LossHead

WIDTH, VOCAB = 96, 1000


@pytest.fixture
def calls(monkeypatch):
    made = []
    for name in ("dl_rmsnorm", "dl_rmsnorm_backward", "dl_head_logprobs",
                 "dl_head_logprobs_backward"):
        monkeypatch.setattr(dh, name, lambda *a, _n=name, **k: made.append(_n))
    return made


def gradients(head, sum_):
    rows = len(sum_)
    t, a = torch.zeros(rows, dtype=torch.int64), torch.zeros(rows)
    head.backward(sum_, t, a, torch.empty(rows, WIDTH), dembed=torch.empty(VOCAB, WIDTH))


def test_backward_takes_the_last_score_only(calls):
    head = LossHead(torch.ones(WIDTH), torch.zeros(VOCAB, WIDTH), 8)
    x, r, s = (torch.zeros(6, WIDTH) for _ in range(3))
    with pytest.raises(RuntimeError):
        gradients(head, x)
    head.score(x)                                        # the stream itself
    gradients(head, x)
    gradients(head, x)                                   # twice, e.g. of two losses
    head.score(x, r, sum_=s)
    gradients(head, s)
    head.score(x, r, sum_=x)                             # in place
    gradients(head, x)
    probe = torch.zeros(6, WIDTH)
    head.score(x, r, sum_=s)
    head.score(probe)                                    # between a step's two halves
    calls.clear()
    with pytest.raises(ValueError):
        gradients(head, s)
    head.score(s[:4])                                    # the same memory, fewer rows
    calls.clear()
    for rows in (6, 3, 5):
        with pytest.raises(ValueError):
            gradients(head, s[:rows])
    with pytest.raises(ValueError):
        gradients(head, s[1:5])
    assert not calls
    gradients(head, s[:4])
    assert calls == ["dl_head_logprobs_backward", "dl_rmsnorm_backward"]


def test_sums_that_score_did_not_keep(calls):
    """Only their number can be told apart then."""
    head = LossHead(torch.ones(WIDTH), torch.zeros(VOCAB, WIDTH), 8)
    x, r = torch.zeros(6, WIDTH), torch.zeros(6, WIDTH)
    head.score(x, r)
    gradients(head, x + r)
    with pytest.raises(ValueError):
        gradients(head, (x + r)[:5])


def test_a_refused_score_leaves_nothing_to_go_by(calls, monkeypatch):
    head = LossHead(torch.ones(WIDTH), torch.zeros(VOCAB, WIDTH), 8)
    x = torch.zeros(6, WIDTH)
    head.score(x)

    def refuse(*a, **k):
        raise dl.DLError(dl.DL_E_INVAL, "dl_head_logprobs")

    monkeypatch.setattr(dh, "dl_head_logprobs", refuse)
    with pytest.raises(dl.DLError):
        head.score(x)
    with pytest.raises(RuntimeError):
        gradients(head, x)


def test_no_rows(calls):
    head = LossHead(torch.ones(WIDTH), torch.zeros(VOCAB, WIDTH), 8)
    head.score(torch.zeros(0, WIDTH))
    gradients(head, torch.zeros(0, WIDTH))
