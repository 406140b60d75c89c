"""The feed-forward sub-block's host side at the edges of its arguments (no
GPU: sizes of workspaces, and calls that a check ends before any launch)."""
import os
import re
import subprocess
import sys

import pytest
import torch

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


def kernel_source(name):
    """The text of a kernel's body in norm.cu."""
    text = open(os.path.join(ROOT, "zero_partitioned_mixed_layout_gb300", "csrc", "norm.cu")).read()
    at = text.index("{", text.index(f" {name}(const __grid_constant__"))
    depth = 0
    for end in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        if depth == 0:
            return text[at:end]
    raise AssertionError(name)


def test_norm_backward_waits_for_its_copies_before_their_memory_is_used_again():
    """A team's last turn, and a team without rows, issue copies that write
    zeros to shared memory; a barrier does not order them, only their thread's
    own wait does, so it comes between the rows and the sums over the block."""
    body = kernel_source("k_norm_bwd_rows")
    last_issue = body.rindex("second(std::false_type{})")
    join = body.index("float4 *const to = s_rows + team", last_issue)
    between = body[last_issue:join]
    assert "copies_done();" in between
    assert between.index("copies_done();") < between.rindex("__syncthreads();")


@pytest.mark.parametrize("name", ["k_norm_fwd_rows", "k_norm_bwd_rows"])
def test_a_staging_kernel_ends_without_copies_under_way(name):
    """After the loop over rows, before the first return: the copies that the
    last turn (or a team without rows) has issued."""
    body = kernel_source(name)
    loop = body.index("{", body.rindex("r < a.rows.rows; r += step"))
    depth = 0
    for end in range(loop, len(body)):
        depth += {"{": 1, "}": -1}.get(body[end], 0)
        if depth == 0:
            break
    after = body[end:]
    assert "copies_done();" in after
    assert "return" not in after[:after.index("copies_done();")]


def test_few_token_rows_are_counted_without_a_sign():
    """Rows of a weight matrix go up to 2^31 - 512, and a block's next row is up
    to 152 * 4 * 8 further: past 2^31, where a signed count would be negative
    and pass for a row in front of the matrix."""
    text = open(os.path.join(ROOT, "zero_partitioned_mixed_layout_gb300", "csrc", "ffn.cu")).read()
    body = text[text.index("k_ffn_tokens(const __grid_constant__ TokenArgs a)"):]
    loop = re.search(r"for \((\w+) n0 = blockIdx.x \* per_block; n0 < (\w+);", body)
    assert loop and loop[1] == "uint32_t"
    assert re.search(rf"const uint32_t {loop[2]} = a\.n;", body)
    assert re.search(r"const uint32_t n = n0 \+ unit;", body)
    most, step = 2 ** 31 - 512, 152 * 4 * 8
    assert most + step < 2 ** 32


@pytest.mark.parametrize("cols", [1, 8, 33, 256, 1001, 1600, 2049, 8192, 8200, 16384, 20001, 40000, 1 << 20])
def test_layer_norm_workspace_for_many_rows_serves_fewer(zp, cols):
    sizes = [zp.zero_layer_norm_workspace_bytes(rows, cols) for rows in range(2000)]
    assert sizes == sorted(sizes)
    assert sizes[-1] <= zp.zero_layer_norm_workspace_bytes(1 << 20, cols)
    # and no row's two sums are without a place while a block may take one row
    assert all(s >= 256 + min(rows, 64) * 2 * cols * 4 for rows, s in enumerate(sizes))


def test_layer_norm_workspace_for_wide_rows_serves_narrow_ones(zp):
    for rows in (1, 5, 100, 153, 761, 1217, 100_000):
        sizes = [zp.zero_layer_norm_workspace_bytes(rows, cols) for cols in range(0, 40_000, 7)]
        assert sizes == sorted(sizes)


@pytest.mark.parametrize("dim,inner", [(1, 1), (8, 8), (64, 256), (1600, 6400), (1001, 2731), (1600, 6401), (13, 8)])
def test_gated_ffn_workspace_for_many_tokens_serves_fewer(zp, dim, inner):
    for backward in (False, True):
        sizes = [zp.zero_gated_ffn_workspace_bytes(m, dim, inner, backward) for m in range(600)]
        assert sizes == sorted(sizes)
    # the backward pass's is enough for the forward
    assert all(zp.zero_gated_ffn_workspace_bytes(m, dim, inner, True) >= zp.zero_gated_ffn_workspace_bytes(m, dim, inner)
               for m in range(600))


def test_a_dropout_draws_from_what_its_fields_are_at_the_call(zp):
    """The struct that a call gets follows the fields, as a new step sets them."""
    d = zp.Dropout(0.25, 5, 7)
    assert (d.p, d.seed, d.offset, d.d_offset) == (0.25, 5, 7, None)
    d.offset += 1
    d.p, d.seed = 0.5, -1
    c = zp.binding._drop_ref(d)._obj
    assert (c.p, c.seed, c.offset, c.d_offset) == (0.5, 2 ** 64 - 1, 8, None)
    with pytest.raises(ValueError):
        d.d_offset = torch.zeros(1, dtype=torch.int64)
    assert d.d_offset is None and zp.Dropout(0.1, 2 ** 64 + 3, -2)._c.offset == 2 ** 64 - 2
