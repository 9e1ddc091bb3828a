"""fa_fwd_paged_chunk at the edges of what fa.h defines: far more tokens than keys, last tiles without a page that can be
read, scores that vanish, scales far apart, and waits that give up."""
import math

import numpy as np
import pytest
import torch

import exact_attention_82_gb300 as fa
import paged_util as pu
from test_gpu_paged_chunk import check, put_back, reference, run_chunk

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status_clean():
    yield
    assert fa.fa_device_status() == fa.FA_OK


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,L,Hkv", [(3841, 462, 1), (6397, 1125, 1), (4117, 475, 2), (6128, 871, 1)])
def test_thousands_of_tokens_more_than_keys(n, L, Hkv, D):
    """Most rows see no key, and the blocks' shares are by far longer than the few tiles of the rows that do: cuts that fall on
    the same tile (on 152 SMs; a replay of the cuts found the sizes).  The workspace holds what an earlier call may have left."""
    c = pu.Cache([L], Hkv, 64, D, seed=n)
    q, cu, d_cu = pu.queries([n], Hkv, D, seed=L)
    ws = torch.full((fa.fa_fwd_paged_chunk_workspace_bytes(1, n, Hkv, Hkv, D) // 4,), 3.0, device="cuda").view(torch.uint8)
    run_chunk(c, q, cu, d_cu, workspace=ws)


# The last tile's only page: pages of a whole tile, and sequences whose last tile has one page.
ONLY_PAGES = [(128, 300), (64, 300), (16, 260), (32, 385), (16, 513)]
