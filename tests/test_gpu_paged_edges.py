"""The paged memory cache's calls at the edges of what they take: values that are not finite or of extreme size, calls
that are refused half way, token ranges that are none.  Against float64 numpy (paged_reference.py)."""
import numpy as np
import pytest
import torch

from mamba_ssd_state_b200 import dart
from tests import paged_reference as ref
from tests.parity import rel_err
from tests.test_gpu_paged import SHAPES, TOL, Pool, attention_inputs, cumulative, ints, memories_of

pytestmark = pytest.mark.gpu
FOUR_BIT = [v for v in SHAPES if v[3] == "mxfp4"]


# ------------------------------------------- 4-bit blocks that are no numbers
@pytest.mark.parametrize("N, P, dtype, cache, H, G", FOUR_BIT)
@pytest.mark.parametrize("lens", [[1], [2], [4], [5], [8], [3, 7]])
@pytest.mark.parametrize("row", [0, 1, 7, 8, 9, 34, 63])
def test_a_scale_of_255_is_nan_for_every_token_that_sees_it(N, P, dtype, cache, H, G, lens, row):
    """Blocks from elsewhere may have codes that are not zero beside the scale byte 255; whichever column holds the
    block and whichever token sees it, even or odd, its readout is NaN."""
    rng = np.random.default_rng(row + sum(lens))
    memories = memories_of(rng, [6] * len(lens), H, N, P, cache, scale=0.5)
    pool = Pool(memories, H, N, P, 4, cache, rng)
    for b in range(len(lens)):
        pool.scales[pool.table_np[b, 0], :, 3, row, (row + b) % (N // 32)] = 255
    T = sum(lens)
    args, args64 = attention_inputs(rng, T, H, G, N, P, dtype)
    for sees in (lambda t: t % 2 == 0, lambda t: t % 2 == 1, lambda t: True):
        see = np.array([bool(sees(t)) for t in range(T)])
        counts = np.where(see, 6, 3).tolist()
        out = dart.dart_sma_paged(*args, cumulative(lens), pool.pages, pool.table, ints(*counts), 1.0, scales=pool.scales)
        dart.dart_sync_status()
        want = ref.sma(*args64, lens, memories, [3] * T)
        assert torch.isnan(out[torch.from_numpy(see).cuda()]).all()
        assert rel_err(out[torch.from_numpy(~see).cuda()], want[~see]) <= TOL if (~see).any() else True
