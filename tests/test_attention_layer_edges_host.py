"""Host-side edges of the attention layer's entry points and of the binding's workspaces (no GPU needed)."""
import pytest


@pytest.fixture(scope="module")
def lib():
    from linear_attention_recurrent_chunked_b200 import build, gdn
    build.build()
    return gdn.load_library()


def test_injection_kinds_of_the_attention_layer(lib):
    """The kinds that withhold a load, their bounds, and nothing beyond them."""
    try:
        for kind in (2, 3):
            assert lib.gdn_debug_inject(kind, 20000) == 0
            assert lib.gdn_debug_inject(kind, 0) == 2
            assert lib.gdn_debug_inject(kind, 1000001) == 2
        for kind in (4, -1):
            assert lib.gdn_debug_inject(kind, 20000) == 2
    finally:
        assert lib.gdn_debug_inject(0, 0) == 0
