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


class OnDevice:
    """What the binding asks a device tensor first."""

    def get_device(self):
        return 0

    def __getattr__(self, name):
        raise AssertionError("looked at %s" % name)


class OtherDevicesStream:
    device_index = 1
    cuda_stream = 0  # a default stream: the same handle on every device


def test_a_stream_of_another_device_is_refused():
    x = OnDevice()
    with pytest.raises(ValueError, match="stream is of device 1"):
        gqa.paged_append(x, x, x, x, x, x, x, stream=OtherDevicesStream())
    with pytest.raises(ValueError, match="stream is of device 1"):
        gqa.paged_attention(x, x, x, x, x, x, stream=OtherDevicesStream())


def test_an_object_with_a_handle_is_a_stream():
    class Handle:
        cuda_stream = 7
    gqa._check_stream(Handle(), 0)
    gqa._check_stream(None, 0)
