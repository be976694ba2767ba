"""The training operators (GPU) where they once went wrong."""
import numpy as np
import pytest
import torch

from selective_state_space_76_amd import AdamW, embedding_bwd
from tests.test_embedding_gpu import bwd_check, tokens_of

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


# few rows in [B, E, L]: on both sides of what products take
@pytest.mark.parametrize("B,L,V,E", [(4096, 3, 60, 40), (1000, 2, 4, 130), (700, 17, 32, 70), (600, 64, 16, 64),
                                     (300, 255, 5, 40), (300, 256, 5, 40), (40, 640, 33, 130), (40, 520, 64, 130)])
@pytest.mark.parametrize("ot", [F32, BF16], ids=["f32", "bf16"])
def test_many_short_rows_of_letters(B, L, V, E, ot):
    for add in (False, True):
        print("case: embed grad letters", B, L, V, E, ot, add, flush=True)
        bwd_check(tokens_of(B, L, V, B + L), V, E, ot, F32, True, 1.5, seed=V, add=add)


@pytest.mark.parametrize("cf,V", [(True, 40), (True, 4), (True, 300), (False, 300)])
@pytest.mark.parametrize("gt", [F32, BF16], ids=["gf32", "gbf16"])
def test_adding_leaves_the_rows_of_other_tokens_alone(cf, V, gt):
    """Bit for bit, a negative zero among them, whatever lies in the gradients."""
    tok = torch.randint(0, V, (2, 700), generator=torch.Generator().manual_seed(V))
    named = torch.arange(V) % 3 == 0
    tok = tok // 3 * 3
    for bad in (False, True):
        print("case: embed grad added", cf, V, gt, bad, flush=True)
        dout = -torch.rand((2, 50, 700) if cf else (2, 700, 50))
        if bad:
            dout[0, 3, 5] = float("nan")
        dw = torch.full((V, 50), -0.0, dtype=gt)
        dw[1::3] = float("nan")
        got = embedding_bwd(tok.to(DEV), dout.to(DEV), V, channels_first=cf, dweight=dw.to(DEV), accumulate=True).cpu()
        bits = torch.int32 if gt == F32 else torch.int16
        assert torch.equal(got.view(bits)[~named], dw.view(bits)[~named])
        occurs = torch.isin(torch.arange(V), tok)
        assert (got[occurs] != 0).all()


def test_a_step_behind_a_kept_graph():
    p = torch.ones(300, device=DEV, requires_grad=True)
    loss = (p * p).sum()
    loss.backward(retain_graph=True)
    AdamW([p]).step()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
