"""The workspace of a sampling call is enough for every smaller one (CPU)."""
import random

import offloaded_expert_slot_amd as oes


def test_workspace_never_falls_as_the_batch_grows():
    for vocab in (1, 100, 4089, 4090, 12289, 32000, 100003, 128256, 200003, 1 << 18, (1 << 20) - 7, 1 << 20):
        last = 0
        for n in range(0, 2200):
            bytes_ = oes.sample_workspace_bytes(n, vocab)
            assert bytes_ >= last, (n, vocab)
            last = bytes_


def test_workspace_never_falls_as_the_vocabulary_grows():
    for n in (1, 7, 48, 64, 65, 81, 82, 128, 700, 2047, 2048, 2049, 5000):
        last = 0
        for vocab in sorted({v for m in range(1, 257) for v in (4096 * m - 8, 4096 * m - 7, 4096 * m - 6)}):
            bytes_ = oes.sample_workspace_bytes(n, vocab)
            assert bytes_ >= last, (n, vocab)
            last = bytes_


def test_workspace_of_random_pairs():
    rng = random.Random(5)
    for _ in range(20000):
        n, vocab = rng.randint(1, 3000), rng.randint(1, 300000)
        less_n, less_vocab = rng.randint(0, n), rng.randint(1, vocab)
        assert oes.sample_workspace_bytes(less_n, less_vocab) <= oes.sample_workspace_bytes(n, vocab), (less_n, less_vocab, n, vocab)
