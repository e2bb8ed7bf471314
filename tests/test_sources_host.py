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


def test_every_kernel_with_an_abort_flag_lets_its_copies_land():
    """Between the barrier that ends the roles and the kernel's last brace the
    flag is asked, in the kernel whose producers may have left before it was
    set."""
    found = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        code = re.sub(r"//[^\n]*", "", open(path).read())
        for body in re.findall(r"__global__ [^;{]*?\{\n(.*?)\n\}\n", code, re.S):
            if "volatile int s_abort" not in body:
                continue
            found += 1
            end = body[body.rindex("tc_fence_before();"):]
            joined = re.search(r"__syncthreads\(\);|cluster_sync\(\);", end)
            asked = re.search(r"if \((s_abort|gave_up)\) let_copies_land\(\);", end)
            assert joined and asked and joined.end() <= asked.start() < end.index("dealloc"), path
    assert found == 7  # NVFP4 and 8-bit linears, single CTAs and pairs; the three of the block linear
