"""Batches that the chunk attention takes and refuses by their size alone (host side)."""
import io_aware_attention_flash_gb300 as fa


def test_places_of_a_batch():
    bytes_of = lambda B: fa.fa_chunk_cache8_workspace_bytes(B, 1, B, 4, 4, 100, 64)  # noqa: E731
    assert bytes_of(2 ** 26) > 0 and bytes_of(2 ** 26 + 1) == 0 and bytes_of(2 ** 28) == 0
