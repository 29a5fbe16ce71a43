"""The paged 4-bit cache at its edges, on a host without a GPU: what calls without work, orders of kernels and index
arithmetic have to keep to."""
import pathlib
import re

import pytest

CSRC = pathlib.Path(__file__).resolve().parent.parent / "block_quantized_weight_quantize_gb300" / "csrc"


@pytest.mark.parametrize("file,kernel", [("qb_kv.cu", "kv_cache_rows_kernel"), ("qb_kv_pages.cu", "kv_pages_copy_kernel")])
def test_writers_of_a_key_cache_let_no_kernel_start_early(file, kernel):
    """kv_scores reads its first key tiles before it waits for the kernel before it, so no kernel that may write a key cache
    starts its successor early."""
    text = (CSRC / file).read_text()
    body = re.search(r"__global__[^;{]*\b%s\(.*?\n}\n" % kernel, text, re.S).group(0)
    assert "pdl_wait();" in body and "pdl_launch_dependents();" not in body
