"""What the serving operators' bindings answer on the host alone (CPU only)."""
import pytest

from mixed_precision_attention_gb300 import _lib, build


@pytest.fixture(scope="module")
def apa():
    build.build()
    import mixed_precision_attention_gb300 as apa
    return apa


@pytest.mark.parametrize("at", range(4))
@pytest.mark.parametrize("x", [2 ** 32 + 1, 2 ** 31, -2 ** 32 + 1, -1, 0])
def test_workspace_sizes_of_counts_past_32_bits(apa, at, x):
    """0, as for every count that the call refuses, not what their low 32 bits would need."""
    sizes = [2, 4, 2, 1]
    assert apa.attention_cache_workspace_bytes(*sizes, 64) > 0
    sizes[at] = x
    assert apa.attention_cache_workspace_bytes(*sizes, 64) == 0


def test_workspace_size_of_a_head_dimension_past_32_bits(apa):
    assert apa.attention_cache_workspace_bytes(2, 4, 2, 1, 2 ** 32 + 64) == 0


def test_the_device_error_names_what_is_reported(apa):
    """A wait that ran out, and pages, slots and lengths in device memory that are out of range."""
    text = _lib.status_string(-7)
    assert all(w in text for w in ("timed out", "page", "slot", "length"))


def test_alignment_errors_name_strides():
    build.build()
    text = _lib.status_string(-8)
    assert "16-byte" in text and "stride" in text
