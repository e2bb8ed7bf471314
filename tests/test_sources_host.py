"""The sources hold no device helper that nothing calls."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "vlaq_quantize_act_b200", "csrc")


def test_every_device_helper_is_called():
    text = {p: open(p).read() for p in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))}
    code = re.sub(r"//[^\n]*", "", "\n".join(text.values()))
    names = set(re.findall(r"__device__ (?:__forceinline__|__noinline__) [\w ]+?[\s*&](\w+)\(", code))
    assert len(names) > 50
    unused = sorted(n for n in names if len(re.findall(rf"\b{n}\b", code)) < 2)
    assert not unused, unused
