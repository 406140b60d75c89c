"""What the attention kernels' sources say where no run could show it."""
import os

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def kernel_source(name):
    """The text of a kernel's body in attention.cu."""
    text = open(os.path.join(ROOT, "zero_partitioned_mixed_layout_gb300", "csrc", "attention.cu")).read()
    at = text.index("{", text.index(f" {name}(const __grid_constant__"))
    depth = 0
    for end in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        if depth == 0:
            return text[at:end]
    raise AssertionError(name)


def test_backward_kernels_wait_before_they_read_what_was_written_before():
    """The statistics are another kernel's, and a launch that was let start
    early sees them only behind a wait of its own: in every CTA, whatever the
    call, before the first read."""
    for name in ("k_attn_dkv", "k_attn_dq"):
        body = kernel_source(name)
        wait = body.index("pdl_wait();")
        line = body[body.rindex("\n", 0, wait) + 1:wait]
        before = body[:wait].rstrip().splitlines()[-1].strip()
        assert line == "    ", name  # (of the kernel's own scope)
        assert before.startswith("//") or before.endswith(";"), name  # (of no condition)
        assert "f.stats" not in body[:wait] and "a.q_offsets" not in body[:wait], name
