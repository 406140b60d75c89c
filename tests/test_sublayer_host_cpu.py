"""The feed-forward sub-block's host side at the edges of its arguments (no
GPU: sizes of workspaces, and calls that a check ends before any launch)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def zp():
    from zero_partitioned_mixed_layout_gb300 import _build
    _build.build()
    import zero_partitioned_mixed_layout_gb300 as zp
    zp.binding._sublayer_lib()
    return zp


def in_child(code):
    """Runs `code` in a process of its own, which a signal may end."""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr[-2000:])
    return r.stdout.split()


def test_layer_norm_backward_of_no_columns(zp):
    """Matrices without columns are empty arrays: a workspace of the header
    alone, and a call that its checks end, not a division by their width."""
    out = in_child(
        "import zero_partitioned_mixed_layout_gb300 as zp\n"
        "so = zp.binding._sublayer_lib()\n"
        "for rows in (0, 1, 4, 5000):\n"
        "    print(zp.zero_layer_norm_workspace_bytes(rows, 0))\n"
        "def bwd(rows, ws, wsb):\n"
        "    return so.zero_layer_norm_backward(None, 0, None, 0, None, 0, None, None, None, 0, None, 0, None, None, 0,\n"
        "                                       None, None, 0, rows, 0, 0, ws, wsb, None)\n"
        "print(bwd(4, 256, 16), bwd(4, 128, 256), bwd(4, None, 256), bwd(0, 256, 16))\n")
    assert out[:4] == ["256"] * 4
    assert out[4:] == ["-5", "-2", "-5", "-5"]  # ZERO_EWORKSPACE, ZERO_EALIGN
