"""What the workspace of the vocabulary loss holds, as its header says: no logits in the
forward; G in the backward, as planes of bf16, rows rounded up to 256, 1 GiB at a time
or 2048 columns if those are more.  No GPU needed."""
import pytest

import nonlinear_rnn_gb300 as nr

GIB = 1 << 30


@pytest.mark.parametrize("dtype,planes", [(0, 3), (1, 1)])
@pytest.mark.parametrize("n,V,d", [(1, 1, 1), (4, 50021, 1024), (64, 50021, 512), (65, 50021, 512), (3001, 10007, 250), (4096, 32768, 512),
                                   (8192, 65536, 1024), (16384, 65536, 1024), (262144, 65536, 1024), (5, 2_200_000, 64)])
def test_the_loss_keeps_what_its_header_says(n, V, d, dtype, planes):
    lib = nr.load()
    forward, backward = (lib.nrnn_vocab_loss_workspace_bytes(n, d, V, dtype, b) for b in (0, 1))
    rows, pitch, columns = -(-n // 256) * 256, -(-d // 8) * 8, -(-V // 256) * 256
    of_g = 3 if dtype == 0 else 2 if n <= 64 else 1
    inputs = 2 * planes * (rows + V) * pitch              # x and W laid out (W only where it has to be)
    # forward: two values for each row and group of column tiles, or warp of the few-rows form
    assert forward <= inputs + 8 * n * max(2 * -(-V // 64), 4 * 76 * 8) + 12 * n + 4096
    whole = 2 * of_g * rows * columns
    one = max(min(whole, GIB), min(2 * of_g * rows * 2048, whole))
    parts = 4 * 2 * 76 * 256 * 256                        # sums of cut tiles
    assert backward <= inputs + one + parts + 4 * rows * pitch + 24 * n + 8192
    if whole <= GIB:
        assert backward >= whole                          # all of rows x V at once
    if n == 8192 and dtype == 1:
        assert whole == GIB
