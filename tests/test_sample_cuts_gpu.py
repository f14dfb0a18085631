"""gc_sample's cuts where the histogram of the weights, whose amounts are
rounded, points to a bin that holds more tokens than a list and ends before
the cut."""

import numpy as np
import pytest
import torch

from test_rows_gpu import check_sample

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,vocab", [(1, 40001), (5, 33000), (320, 9000)])
@pytest.mark.parametrize("top_k", [0, 7000])
def test_top_p_ends_after_thousands_of_equal_values(rows, vocab, top_k):
    # 5000 equal tokens whose weight lies just above half a unit of 2^-14, the
    # unit in which the largest are counted: together they count for 0.15 more
    # than they weigh.  100 lighter ones weigh 0.25, and top-p ends after 40.
    x64 = np.full((rows, vocab), -30.0)
    for r in range(rows):
        at = np.random.default_rng(r).permutation(vocab)
        x64[r, at[0]] = 0.0
        x64[r, at[1:5001]] = np.log((16200.5 + 0.05) / 16384)
        x64[r, at[5001:5101]] = -6.0 - 0.001 * np.arange(100)
    x = torch.from_numpy(x64.astype(np.float32)).cuda()
    x64 = x.double().cpu().numpy()
    u = torch.full((rows, vocab), 0.01, device="cuda")
    params = []
    for r in range(rows):
        at = np.argsort(-x64[r], kind="stable")
        w = np.exp(x64[r][at])
        upto = np.cumsum(w)
        total = upto[top_k - 1] if top_k else upto[-1]
        params.append((1.0, top_k, (upto[5039] + upto[5040]) / 2 / total, 0.0))
        # a token past the cut wins if it is kept: 16.6 - 6.1 against -1.5
        u[r, int(at[5080])] = 1 - 2.0 ** -24
    check_sample(x, x64, u, params, vocab)
