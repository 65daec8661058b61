"""How kernels read what another call of the library may have written just
before them on the stream: block tables, lengths and slots (pa_plan_append,
pa_tree_accept), rotated keys (pa_norm_rope_and_cache).  With programmatic
launches a kernel can be resident while the one before it still runs.  Its
wait orders ordinary loads; the read-only path (__ldg) is for data that nobody
writes while the kernel is resident, and its loads may be moved across the
wait.  No GPU needed."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_354_b200", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def test_tree_calls_read_what_a_step_writes_with_ordinary_loads():
    for name in ("pa_tree.cu", "pa_plan.cu", "pa_norm_rope.cu"):
        text = source(name)
        assert [x for x in re.findall(r"__ldg\(([^;]*);", text) if "weight" not in x] == []
        assert "ld.global.nc" not in text and "__restrict__" not in text


def test_what_the_read_only_path_reads_is_written_before_its_reader_starts():
    """The decodes and the cache write take tables, lengths, slots and new keys
    through the read-only path.  A kernel that writes one of them does not let
    the next one start early, unless that one is its own call's second kernel
    (a large plan's slots) or nothing of the kind is written (no k_out)."""
    assert [line.split("//")[0].strip() for line in source("pa_plan.cu").splitlines() if "pdl_trigger" in line] == [
        "if (!kSlots && a.num_slots > 0) pdl_trigger();"]
    assert [line.strip() for line in source("pa_norm_rope.cu").splitlines() if "pdl_trigger" in line] == [
        "if (a.k_out == nullptr) pdl_trigger();"]
