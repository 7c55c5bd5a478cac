"""Rules that the CUDA sources keep."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_sparse_attention_plan_gb300", "csrc")


def sources():
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh", ".h")):
            with open(os.path.join(CSRC, name)) as f:
                yield name, re.sub(r"//[^\n]*", "", f.read())


def test_overlapping_launches_read_nothing_through_the_read_only_path():
    """A kernel that launch_after starts may be resident while the one ahead of
    it, or the caller's, still writes what it is given: its loads are plain ones,
    behind the wait.  Only kernels launched the ordinary way may use __ldg."""
    seen = 0
    for name, text in sources():
        ordinary = "launch_after(" not in text and "<<<" in text
        if not ordinary:
            assert not re.search(r"__ldg\b|ld\.global\.nc|__restrict__", text), name
            seen += "launch_after(" in text
    assert seen >= 7


def test_kernels_that_overlap_wait_before_they_read():
    """next_may_launch() and wait_for_previous() come as a pair, in every file
    whose kernels launch_after starts."""
    for name, text in sources():
        if name != "bsa_launch.h" and "launch_after(" in text:
            assert text.count("next_may_launch();") == text.count("wait_for_previous();") > 0, name


def test_shared_memory_limits_are_constants():
    """A kernel's limit of dynamic shared memory belongs to the kernel, which host
    threads share: set to what one call needs, it may be too small for another's
    launch.  Every setting is a constant expression."""
    found = 0
    for name, text in sources():
        for m in re.finditer(r"cudaFuncAttributeMaxDynamicSharedMemorySize,\s*([^;]*?)\);", text):
            found += 1
            value = m.group(1).replace("(int)", "")
            if re.fullmatch(r"\w+", value) and not value.startswith("k"):  # a variable: what it is set to
                value = re.search(r"int %s = ([^;]*);" % value, text).group(1)
            names = [w for w in re.findall(r"[A-Za-z_]\w*", value) if w not in ("sizeof", "int")]
            assert any(w.startswith("k") for w in names) and "n" not in names, (name, value)
    assert found >= 5


def test_copies_of_the_prompt_kernel_are_awaited_at_its_end():
    """A wait may give up when the copies have long been requested and their requester is done: what waits for them
    stands behind the CTA's last barrier, ahead of nothing but the release of tensor memory."""
    text = dict(sources())["bsa_prompt_attn.cu"]
    body = text[text.index("prompt_kernel("):text.index("prompt_schedule_kernel")]
    end = body[body.rindex("__syncthreads();"):]
    assert "abort_flag" in end and "drain_copies" in end and body.count("drain_copies") == 1
    assert "return" not in body
