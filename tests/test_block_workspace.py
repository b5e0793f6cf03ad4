"""What the feed-forward block's workspace holds.  No GPU needed."""
import pytest

import nonlinear_rnn_gb300 as nr


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("n,d,f", [(32768, 1024, 4096), (1501, 250, 683), (100, 16, 24)])
def test_a_forward_that_keeps_nothing_takes_no_room_for_the_gradient(n, d, f, dtype):
    """The planes of m, copies of the operands (of tensors that are not used where they lie),
    sums of cut tiles, and a few alignments: not what a gradient would take besides."""
    planes, pd, pf = 1 if dtype else 3, -(-d // 8) * 8, -(-f // 8) * 8
    m, copies, parts = 2 * planes * n * pf, 2 * planes * (n * pd + 2 * f * pd + d * pf), 4 * 2 * 76 * 256 * 256
    size = nr.load().nrnn_gated_mlp_workspace_bytes(n, d, f, dtype, 0)
    assert m + copies < size <= m + copies + parts + 8 * 256
