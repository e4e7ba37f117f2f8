"""qmm_sample's workspace follows the vocabulary (a row of 100 tokens needs no list of 16384)."""
import block_quantized_matmul_amd as qmm


def test_small_vocabularies_need_little():
    W = qmm.qmm_sample_workspace_bytes
    assert W(4096, 100) < 120 << 20
    before = 0
    for vocab in (1, 15, 16, 17, 100, 1000, 8191, 8192, 8193, 16384, 16385, 40000, 524287):
        need = W(3, vocab)
        assert need >= before and need % 8 == 0 and need >= 3 * 8 * min(vocab, 16384)
        before = need
