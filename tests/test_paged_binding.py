"""The Python binding of the paged cache, without a GPU."""
import pytest

import attention_gqa_b200 as gqa


@pytest.fixture(scope="module", autouse=True)
def built():
    from attention_gqa_b200 import build
    build.build()


class Size:
    """A size that its owner may change, such as a 0-d tensor."""

    def __init__(self, value):
        self.value = value

    def __int__(self):
        return self.value


def test_the_workspace_query_follows_what_its_arguments_hold_now():
    window = Size(128)
    assert gqa.paged_attention_workspace_bytes(1, 1, 8192, window) == 0
    window.value = 0
    assert gqa.paged_attention_workspace_bytes(1, 1, 8192, window) > 0


@pytest.mark.parametrize("n", [1, 2, 5, 40])
def test_a_workspace_of_the_largest_batch_serves_smaller_ones(n):
    sizes = [gqa.paged_attention_workspace_bytes(b, n, 8192) for b in (1, 2, 63, 500, 1023, 1024, 3000)]
    assert sizes == sorted(sizes) and sizes[0] > 0
