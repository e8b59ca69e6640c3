"""Edges of the verify-step operators that show without a GPU."""
import pytest

from adapter_lora_bgmv_amd import binding as B


@pytest.mark.parametrize("code", [B.LORA_F32, B.LORA_BF16])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 100])
def test_scores_take_at_most_128_chunks_a_row(n, code):
    """The join has places for 128 chunks of a row; a record of 32 alternatives
    is 16 + 8 x 32 bytes, the counters in front take 256 a 64 rows."""
    for V in [(1 << 20) - i for i in range(9)] + [(1 << 19) + 1, 131072, 300000]:
        need = B.lora_token_logprobs_workspace_bytes(code, V, n, 32)
        chunks = (need - (4 * n + 255) // 256 * 256) / n / (16 + 8 * 32)
        assert chunks == int(chunks) and 2 <= chunks <= 128, (V, chunks)
