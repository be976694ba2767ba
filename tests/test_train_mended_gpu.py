"""The training operators (GPU) where they once went wrong."""
import numpy as np
import pytest
import torch

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
