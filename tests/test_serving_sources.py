"""What the sources of the serving kernels must not do, whatever their results."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "precision_causal_attention_block_gb300", "csrc")
FILES = ["paged.cuh", "rope.cu", "cache.cu", "attend.cuh", "attn_cache.cu", "attn_cache_rows.cu"]


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", FILES)
def test_inputs_are_not_read_as_read_only_data(name):
    """Programmatic dependent launch starts a kernel before the one that writes its
    inputs has ended: read-only loads (and pointers that let the compiler make them)
    would ask for data that nobody writes while the kernel lives."""
    code = _code(name)
    assert not re.search(r"__ldg\b|\.nc\b|__restrict__|__restrict\b", code)


def test_every_kernel_waits_for_the_one_before():
    for name in FILES[1:]:
        code = _code(name)
        # (launch bounds may hold parentheses)
        for m in re.finditer(r"__global__ void __launch_bounds__", code):
            body = code[m.start():]
            end = body.find("__global__ void", 1)
            body = body[:end] if end > 0 else body
            assert "wait_for_previous();" in body, (name, body[:120])


@pytest.mark.parametrize("name", ["attn_cache.cu", "attn_cache_rows.cu"])
def test_products_in_flight_end_before_their_memory_goes(name):
    """A CTA whose waits run out frees its tensor memory and exits: the issuer's way out
    commits what it issued to a barrier and waits there, with a limit."""
    code = _code(name)
    failed = [code[m.end():m.end() + 400] for m in re.finditer(r"if \(!ok\) \{", code)]
    assert any(re.search(r"tc_commit(_w)?\(smem_u32\(&sm\.drained\)\);.*"
                         r"mbar_wait_w\(smem_u32\(&sm\.drained\), 0\);", f, re.S) for f in failed)
    assert "mbar_init(smem_u32(&sm.drained), 1);" in code
