"""Kernels launched as programmatic dependents start while the kernel before
them may still be writing their inputs. PTX allows non-coherent loads (__ldg,
ld.global.nc) only of data that is read-only as long as the kernel lives, so
the files of those kernels hold none."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kv_cache_02_b200", "csrc")


def code(path):
    """The source without its comments."""
    return re.sub(r"//[^\n]*", "", open(path).read())


def test_dependents_read_nothing_non_coherently():
    files = [f for f in glob.glob(os.path.join(CSRC, "*.cuh")) if "grid_dep_wait()" in code(f)]
    names = {os.path.basename(f) for f in files} - {"common.cuh"}
    assert names >= {"decode.cuh", "decode_wide.cuh", "decode_scores.cuh", "decode_mxfp4.cuh", "evict.cuh", "mxfp4.cuh",
                     "norm_rope.cuh", "prompt_scores.cuh", "kv_proj.cuh"}
    for f in files:
        assert not re.search(r"__ldg\s*\(|\.nc\b", code(f)), os.path.basename(f)


def test_kernels_with_non_coherent_loads_are_launched_without():
    """The other files' kernels go out as ordinary launches: pdl is false wherever they are named."""
    host = "".join(code(f) for f in glob.glob(os.path.join(CSRC, "*")))
    for name in ("kv_append_kernel", "kv_append_int8_kernel", "kv_write_prompt_kernel", "kv_write_prompt_varlen_kernel",
                 "meanpool_vec_kernel", "meanpool_scalar_kernel"):
        calls = re.findall(r"launch_kernel\([^;]*?\b%s\b[^;]*?,\s*(true|false)," % name, host)
        assert calls and set(calls) == {"false"}, name
    for f in ("prefill.cuh", "prefill_pair.cuh"):
        text = code(os.path.join(CSRC, f))
        assert "__ldg" in text and "ProgrammaticStreamSerialization" not in text
        assert not re.search(r"launch_kernel\([^;]*,\s*true,", text), f
