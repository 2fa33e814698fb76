"""The long-context operators' size functions at the limits of their arguments.  Nothing here launches a kernel."""
from test_step_host import lib  # noqa: F401


def test_key_weights_workspace_out_of_range(lib):
    """What a call refuses needs no workspace: 0."""
    ws = lib.mla_key_weights_workspace_bytes
    assert ws(65535, 64, 128, 100) == 64 * 65535 * 100 * 4 and ws(1, 64, 128, 1 << 30) == 64 << 32
    assert ws(65536, 64, 128, 100) == 0
    assert ws(1, 64, 128, (1 << 30) + 1) == 0
    assert ws(1, 64, 128, 63) == 0                          # a table narrower than the drafts
    assert ws(1, 64, 128, 64) == 64 * 64 * 4
