"""The output head where the other tests' sizes do not reach: past each
variant's threshold, several turns of a workgroup, and a Head's calls mixed
with captured ones.  Tolerances are those derived in test_head_gpu."""
import pytest
import torch

from checkpoint_averaging_amd import dlmerge as dl
from checkpoint_averaging_amd.head import Head
from tests import test_head_gpu as hg
from tests import test_head_path_gpu as hp

pytestmark = pytest.mark.gpu

DEV = "cuda"


def test_captured_score_replays_after_larger_eager_ones():
    """A score of few rows captured, then eager ones of more (the product needs
    more workspace for these) and tensors that fill what may have been freed:
    the replay gives the eager bits and touches nothing else."""
    global_, _ = hp.merged()
    head, other = Head(hp.LAYOUT, global_, 600), Head(hp.LAYOUT, global_, 20)
    needs = [dl.dl_matmul_workspace_bytes(r, hp.VOCAB, hp.WIDTH) for r in (20, 600)]
    assert needs[0] < needs[1]
    x, r, t = hp.stream(20, 1)
    head.score(x, r, t, top_k=3)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a = head.score(x, r, t, top_k=3)
        logits, lps = a.logits.clone(), a.logprobs.clone()
    at = head._product_ws.data_ptr()
    for k in range(4):
        xb, rb, tb = hp.stream(600, 70 + k)
        head.score(xb, rb, tb)
        assert head._product_ws.data_ptr() == at
        others = [torch.full((n,), 7.0, device=DEV) for n in (needs[0] // 4, needs[1] // 4)]
        x2, r2, t2 = hp.stream(20, 50 + k)
        x.copy_(x2)
        r.copy_(r2)
        t.copy_(t2)
        torch.cuda.synchronize()
        g.replay()
        b = other.score(x2, r2, t2, top_k=3)
        torch.cuda.synchronize()
        hg.same_bits(hg.bits(logits), hg.bits(b.logits), "logits")
        hg.same_bits(hg.bits(lps), hg.bits(b.logprobs), "logprobs")
        assert all(bool((o == 7.0).all()) for o in others)
