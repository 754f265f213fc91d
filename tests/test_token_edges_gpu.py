"""GPU tests of the token operators at the edges of their ranges.  The references
and the counting of roundings are those of test_token_ops_gpu.py."""
import numpy as np
import pytest

from conftest import gpu_available
from test_token_ops_gpu import _check_grad, _draw_tokens

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]


@pytest.mark.parametrize("n", [65536 * 64, 65536 * 64 + 1, 5_000_003])
def test_grad_more_tokens_than_merging_workgroups_take_at_once(n):
    """65536 workgroups of 64 tokens: the last of them, one token more, and
    workgroups that take a second turn."""
    import torch

    import dlrm_embedding_bag_amd as fw
    rng = np.random.default_rng(n)
    rows, dim = 3000, 2
    tok = _draw_tokens(rng, n, rows, "hot")
    g = rng.standard_normal((n, dim)).astype(np.float32)
    td, gd = torch.from_numpy(tok).cuda(), torch.from_numpy(g).cuda()
    got = fw.emb_lookup_grad(gd, td, rows)
    _check_grad(got, g.astype(np.float64), tok, rows, 1.0, "f32")
    assert torch.equal(got, fw.emb_lookup_grad(gd, td, rows))
