"""What the serving kernels do before the wait for the kernel in front of them, which writes their
inputs: nothing with those.  Their bodies are cut out of the sources by their braces."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "precision_causal_attention_block_gb300", "csrc")
FILES = ["rope.cu", "cache.cu", "attend.cuh", "attn_cache.cu", "attn_cache_rows.cu", "pages.cu",
         "attn_prefix.cu", "attn_prefix_rows.cu"]
# reads through a pointer of the arguments, or of one of them; what reads by itself
READS = (r"\bg\.\w+(\[[^\]]*\])?\[", r"[=(,;{}&|!?:<>+-]\s*\*\s*g\.", r"\b[kv]_codes\[", r"__ldcg|\bld_|\bcopy16|cp_async|tma_load",
         r"\b(check_offsets|doc_range|find_block|reads_for_all|seq_work|make_plan|shares|load_queries|report|"
         r"renumber|copy_units|eight_counts)\s*[(<]", r"\bRun\s+\w+\(", r"reinterpret_cast<const [^>]*>\((?!smem|sm\b)")


def _closed(code, at, pair="{}"):
    """Index behind the bracket that closes the one at code[at]."""
    depth = 0
    for i in range(at, len(code)):
        depth += (code[i] == pair[0]) - (code[i] == pair[1])
        if depth == 0:
            return i + 1
    raise AssertionError("unbalanced")


def _kernels(name):
    """(name, body) of each __global__ function."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    for m in re.finditer(r"__global__\s+void\s+", code):
        at = m.end()
        bounds = re.match(r"__launch_bounds__\s*\(", code[at:])
        if bounds:
            at = _closed(code, at + bounds.end() - 1, "()")
        head = re.match(r"\s*(\w+)\s*\(", code[at:])
        args = _closed(code, at + head.end() - 1, "()")
        begin = code.index("{", args)
        assert not code[args:begin].strip()
        yield head[1], code[begin:_closed(code, begin)]


def _before_the_wait(body):
    """What runs before it: lambdas are taken out, and come back by their calls."""
    lambdas = {}
    while m := re.search(r"\bauto (\w+) = \[[^\]]*\]\s*\(", body):
        args = _closed(body, m.end() - 1, "()")
        begin = body.index("{", args)
        end = _closed(body, begin)
        lambdas[m[1]] = body[begin:end]
        body = body[:m.start()] + body[end:]
    assert "wait_for_previous();" in body
    text = body[:body.index("wait_for_previous();")]
    for _ in lambdas:
        for name, inner in lambdas.items():
            text = re.sub(rf"\b{name}\(", lambda _: inner + "(", text)
    return text


@pytest.mark.parametrize("name", FILES)
def test_inputs_wait_for_the_kernel_in_front(name):
    found = 0
    for kernel, body in _kernels(name):
        text = _before_the_wait(body)
        for pattern in READS:
            assert not re.search(pattern, text), (name, kernel, re.search(pattern, text)[0])
        found += 1
    assert found


def test_a_read_before_the_wait_is_seen():
    """The search finds what it looks for, in every kernel: the same bodies without their wait's
    place, as if it stood at the end."""
    for name in FILES:
        for kernel, body in _kernels(name):
            text = _before_the_wait(body.replace("wait_for_previous();", "", 1)[:-1] + "wait_for_previous();}")
            assert any(re.search(p, text) for p in READS), (name, kernel)
