"""The windowed backward's workspace as include/fa.h states it: 16-byte aligned, nothing more."""
import pytest

from exact_io_aware_32_gb300 import build, fa
from test_rope_window_refusals_host import A, WORKSPACE, accepted, no_gpu, window


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return fa.load()


def test_workspace_of_16_bytes_alignment_is_taken():
    no_gpu()
    need = fa.fa_bwd_window_workspace_bytes(2, 4, 2, 100, 200, 64, 50, 4)
    for at in (16, 32, 48, 128, 240, 256):
        assert accepted(window(True, workspace=10 * A + at, workspace_bytes=need)), at


@pytest.mark.parametrize("at", [1, 2, 4, 8, 12, 24, 136, 255])
def test_less_aligned_workspace_is_refused(at):
    assert window(True, workspace=10 * A + at) == WORKSPACE
