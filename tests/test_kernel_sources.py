"""What the kernels' sources have to keep to that no run can show."""
import os
import re

import kv_cache_quantize_b200 as kvq

CSRC = os.path.join(os.path.dirname(kvq.__file__), "csrc")


def test_attention_reads_only_constants_through_the_read_only_path():
    """__ldg is for data that nobody writes while the kernel lives.  These kernels may start while the one before them
    still runs, and that one may write lengths, tables, offsets of sequences and queries: only the caches' scales and
    offsets, which no kernel writes, may be read so."""
    seen = 0
    for name in ("attention_common.cuh", "attention_prompt.cuh", "attention_shared.cuh"):
        with open(os.path.join(CSRC, name), encoding="utf-8") as f:
            text = f.read()
        assert "ld.global.nc" not in text
        for arg in re.findall(r"__ldg\(([^;]*)", text):
            seen += 1
            assert re.match(r"(sk|a\.(scale|offset)_[kv]) \+", arg), (name, arg)
        # the one short name among them
        assert all("a.scale_k" in line for line in re.findall(r"\* sk = [^;]*;", text))
    assert seen
