"""The loss of one or two tokens without a GPU: its blocks, one to a piece of
the vocabulary, are no more than run at once."""
import pytest

from pipeline_schedule_simulation_gb300 import binding as B
from pipeline_schedule_simulation_gb300 import stage as S  # noqa: F401  (declares the entry points)

SMS, SM_BYTES = 152, 228 * 1024  # what the library takes where it finds no GPU; shared memory of an SM
P = 1 << 20  # stands for an aligned pointer; never followed


def _pieces(T, V, H):
    """The least and the most number of pieces that the workspace is for: 8 bytes for each piece and token, then 4 for
    each token, each rounded up to 256."""
    n = B.LIB.pp_stage_head_forward_workspace(P, H, P, H, T, V, H) - 256
    return (n - 255) // (8 * T), n // (8 * T)


@pytest.mark.parametrize("T,V,H", [(1, 128000, 2048), (1, 128000, 12288), (1, 131072, 16384), (2, 131072, 4096),
                                   (2, 131072, 7168), (2, 131072, 8192), (1, 32000, 16384)])
def test_blocks_of_few_tokens_run_at_once(T, V, H):
    import torch
    if torch.cuda.is_available():
        pytest.skip("the number of SMs is the GPU's")
    # a block keeps its tokens in 32 bits; 1 KB more is the SM's and 128 bytes are the block's sums
    at_once = SMS * min(4, SM_BYTES // (4 * T * H + 1024 + 128))
    least, most = _pieces(T, V, H)
    assert least <= at_once and most > at_once // 2
