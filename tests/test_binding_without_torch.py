"""The conv binding takes raw device addresses and stream handles from programs that do not have torch."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys
sys.modules["torch"] = None  # an import of it fails
import microscaling_quantized_convolution_mx_amd as mx
d = mx.desc(32, 32, 32, 4, 4, 3, 3)
for stream in (0, 0x7000):
    try:
        mx.mx_conv_fwd(d, mx.mx_qtensor(), mx.mx_qtensor(), None, stream=stream)  # refused on the host
    except mx.MxError as e:
        assert e.status == -1, e.status
    else:
        raise SystemExit("not refused")
print("ok")
"""


def test_raw_addresses_and_handles():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr
