"""CPU tests of arguments that the binding has to refuse by itself."""
import pytest

from exact_attention_forward_tiled_gb300 import api


def test_prefix_without_pages():
    """A length but no pages: refused, not run without the prefix."""
    with pytest.raises(ValueError, match="prefix_pages"):
        api.attention_forward_prefix(None, None, None, 5, None, None)
    with pytest.raises(ValueError, match="negative"):
        api.attention_forward_prefix(None, None, None, -1, None, None)
