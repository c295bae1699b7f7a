"""Rules that the kernels of the e4m3 operators keep because they may start while the kernel before
them in the stream still runs. What breaks them need not show in a run, so the sources are read."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = sorted(glob.glob(os.path.join(ROOT, "post_weight_quantization_18_b200", "csrc", "fp8*.cu*")))


def code_of(path):
    """The file without its comments."""
    return re.sub(r"//[^\n]*", "", open(path).read())


def kernels():
    """(file, text from one __global__ to the next) of every kernel."""
    for path in SOURCES:
        for part in code_of(path).split("__global__")[1:]:
            yield os.path.basename(path), part


def test_the_sources_are_there():
    assert len(SOURCES) >= 8 and len(list(kernels())) >= 8


def test_tensor_memory_comes_before_the_next_kernels_start():
    """A kernel that holds no tensor memory yet must not let the next one start: that one could take the
    tensor memory of an SM and then wait for this kernel, which waits for tensor memory."""
    found = 0
    for name, text in kernels():
        if "tcgen05.alloc" not in text:
            continue
        found += 1
        at = text.find("let_next_kernel_start()")
        assert at < 0 or at > text.index("tcgen05.alloc"), name
    assert found == 3


def test_no_read_only_loads():
    """Inputs may still be written by the kernel before while this one is resident, so nothing may promise
    the compiler that they do not change: no __restrict__, __ldg or ld.global.nc."""
    for path in SOURCES:
        found = re.findall(r"__restrict__|__ldg|\.nc\b", code_of(path))
        assert not found, (os.path.basename(path), found)
