"""fa_fwd_paged_chunk where there is no GPU."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CALL = """
import exact_attention_82_gb300 as fa
need = fa.fa_fwd_paged_chunk_workspace_bytes(1, 4, 2, 1, 128)
at = [0x10000000 * (i + 1) for i in range(11)]  # never read: nothing is launched
for _ in range(2):
    rc = fa.fa_fwd_paged_chunk_raw(*at[:10], 1, 4, 2, 1, 128, 0.1, 256, 4, 8, 64, at[10], need, 0)
    print(rc, fa.fa_strerror(rc))
"""


def test_a_failure_is_named_for_what_it_is():
    """Both calls say what went wrong (no device, or no driver), not that the kernel cannot be launched.  In a process of its
    own that sees no device, so that the made-up addresses reach none."""
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="", PYTHONPATH=ROOT)
    out = subprocess.run([sys.executable, "-c", CALL], env=env, capture_output=True, text=True, timeout=600, check=True).stdout.splitlines()
    assert len(out) == 2
    for line in out:
        assert line.startswith("-7 CUDA error: ") and ("device" in line or "driver" in line), line
