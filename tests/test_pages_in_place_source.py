"""The page update reads words that it may itself write: by its source.

With outputs in place the kernel writes seq_lens (or new_lens) and free_count.  ``__ldg`` is a load by way of the
non-coherent path, for words that nobody writes while the kernel runs."""
import pathlib

SOURCE = pathlib.Path(__file__).resolve().parents[1] / "sparse_attention_paged_dsa_gb300" / "csrc" / "pages_kernel.cu"


def test_no_non_coherent_loads():
    assert "__ldg" not in SOURCE.read_text() and "ld.global.nc" not in SOURCE.read_text().replace("no ld.global.nc", "")
