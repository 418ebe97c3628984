"""The binding imports, and checks its arguments, on a torch that lacks the private
name by which it asks for a device's stream."""
import os
import subprocess
import sys
import textwrap


def run(code):
    r = subprocess.run([sys.executable, "-c", textwrap.dedent(code)], capture_output=True, text=True,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr[-2000:]


def test_without_the_raw_stream_query(lib_path):
    run("""
        import torch
        if hasattr(torch._C, "_cuda_getCurrentRawStream"):
            del torch._C._cuda_getCurrentRawStream
        import normalisation_rope_transformers_gb300 as nrt

        x = torch.zeros(2, 5, 64)
        for groups, what in ((7, "divide"), (8, "CUDA")):
            try:
                nrt.group_norm(x, groups)
            except ValueError as e:
                assert what in str(e), e
            else:
                raise AssertionError("not refused")

        # a launch then takes the stream that torch.cuda.current_stream names
        class Stream:
            cuda_stream = 1234
        asked, got = [], []
        torch.cuda.current_device = lambda: 0
        torch.cuda.current_stream = lambda device=None: asked.append(device) or Stream
        nrt._launch(0, lambda *args: got.append(args) or 0, "a")
        assert asked == [0] and got == [("a", 1234)], (asked, got)
    """)
