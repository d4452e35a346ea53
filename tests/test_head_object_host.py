"""The Head's own rules, on the CPU: the library's calls are replaced by ones
that record their arguments, so nothing is launched."""
import pytest
import torch

from checkpoint_averaging_amd import dlhead as dh
from checkpoint_averaging_amd import dlmerge as dl
from checkpoint_averaging_amd import synth
from checkpoint_averaging_amd.head import Head

WIDTH, VOCAB = 96, 1000
LAYOUT = synth.Layout("small", (("embed", VOCAB * WIDTH), ("final_norm.weight", WIDTH)))


@pytest.fixture
def calls(monkeypatch):
    """(name, arguments) of each library call that would have launched."""
    made = []

    def record(module, name):
        monkeypatch.setattr(module, name, lambda *a, **k: made.append((name, a, k)))

    record(dl, "dl_matmul_f32")
    for name in ("dl_rmsnorm", "dl_w4_quantize", "dl_w4_matvec", "dl_logprobs"):
        record(dh, name)
    return made


def products(calls):
    return [k for name, _, k in calls if name == "dl_matmul_f32"]


@pytest.mark.parametrize("order", [(4, 300, 1000), (1000, 4, 300)], ids=["growing", "shrinking"])
def test_score_keeps_one_product_workspace(calls, order):
    """The need grows with the rows here (384 KiB for 4, more for 300 and 1000),
    and every call has the same memory, which no later call gives back: a call
    captured into a graph keeps its address."""
    head = Head(LAYOUT, torch.zeros(LAYOUT.n_params), max_rows=1000)
    for rows in order:
        head.score(torch.zeros(rows, WIDTH))
    needs = [dl.dl_matmul_workspace_bytes(r, VOCAB, WIDTH) for r in order]
    assert len(set(needs)) == 3
    made = products(calls)
    assert len({k["workspace"].data_ptr() for k in made}) == 1
    for k, need in zip(made, needs):
        assert k["workspace"].numel() * k["workspace"].element_size() >= need
        # the product's plan goes by the bytes it is told of: those of its own rows,
        # whatever the head could hold and whatever ran before
        assert k["workspace_bytes"] == need


@pytest.mark.parametrize("top_k", [-1, dh.DL_MAX_TOP + 1])
@pytest.mark.parametrize("rows", [1, 4])
def test_head_refuses_alternatives_before_any_launch(calls, rows, top_k):
    """The same error for any number of rows, with the last answer still in the buffers."""
    head = Head(LAYOUT, torch.zeros(LAYOUT.n_params), max_rows=4)
    head.publish()
    calls.clear()
    for call in (head.score, head.answer):
        with pytest.raises(ValueError, match="top_k"):
            call(torch.zeros(rows, WIDTH), top_k=top_k)
    assert not calls
    few = synth.Layout("few", (("embed", 5 * WIDTH), ("final_norm.weight", WIDTH)))
    head = Head(few, torch.zeros(few.n_params), max_rows=4)
    with pytest.raises(ValueError, match="top_k"):
        head.score(torch.zeros(rows, WIDTH), top_k=6)                # of five tokens
    assert not calls
    head.score(torch.zeros(rows, WIDTH), top_k=5)
    assert [name for name, _, _ in calls] == ["dl_rmsnorm", "dl_matmul_f32", "dl_logprobs"]


def test_head_takes_its_views_from_the_elements_in_order():
    """A flat vector seen as a matrix is the same vector; one with gaps has no
    views that the kernels could read."""
    n = LAYOUT.n_params
    flat = torch.arange(n, dtype=torch.float32)
    for shape in ((n,), (n // 2, 2), (1, n)):
        head = Head(LAYOUT, flat.view(shape), max_rows=4)
        assert torch.equal(head.embed, flat[:VOCAB * WIDTH].view(VOCAB, WIDTH))
        assert torch.equal(head.weight, flat[VOCAB * WIDTH:])
        assert head.weight.data_ptr() == flat.data_ptr() + 4 * VOCAB * WIDTH
    with pytest.raises(ValueError, match="flat"):
        Head(LAYOUT, torch.zeros(2 * n)[::2], max_rows=4)
