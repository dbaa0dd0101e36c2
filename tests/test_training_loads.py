"""Which loads the training kernels take (no GPU: the sources are read as text). The read-only path
(`ld.global.nc`, __ldg, load_cols) is for memory that nothing writes while a kernel runs, and the
compiler may move such loads; where that does not hold, they have to be coherent."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "hashed_head_gram_gb300", "csrc")


def body(file, name):
    """The braces after the first `name(` of the file that a definition follows."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, file)).read())
    for m in re.finditer(re.escape(name) + r"\(", text):
        at, depth = m.end(), 1
        while depth:
            depth += {"(": 1, ")": -1}.get(text[at], 0)
            at += 1
        rest = text[at:].lstrip()
        rest = rest[len("const"):].lstrip() if rest.startswith("const") else rest
        if rest.startswith("{"):
            end, depth = 1, 1
            while depth:
                depth += {"{": 1, "}": -1}.get(rest[end], 0)
                end += 1
            return rest[:end]
    raise AssertionError(f"{name} is not defined in {file}")


READ_ONLY = re.compile(r"__ldg\(|load_cols<|\.nc\b")


@pytest.mark.parametrize("kernel", ["rowgrad_sum_kernel", "rowgrad_join_kernel"])
def test_kernels_scheduled_early_read_coherently(kernel):
    # the gradient (x[k].load) is the caller's and complete; order, sign and parts are written by the
    # kernels ahead, beside which these already run
    text = body("pg_rowgrad.cu", kernel)
    assert "grid_dep_wait()" in text
    assert not READ_ONLY.search(text)


def test_the_join_reads_parts_after_its_wait():
    text = body("pg_rowgrad.cu", "rowgrad_join_kernel")
    before = text[:text.rindex("grid_dep_wait()")]
    assert "a.parts" not in before[:before.index("auto add =")] and before.count("add(") == 0
    assert READ_ONLY.search(body("pg_vec.h", "load_now")) is None


@pytest.mark.parametrize("name", ["norm_part", "scale_rows"])
def test_orthogonalize_reads_g_coherently(name):
    # the result may lie in G's place, written by the launch that reads G
    assert not READ_ONLY.search(body("pg_ortho.cu", name))


def test_orthogonalize_wide_loads_are_coherent():
    text = open(os.path.join(CSRC, "pg_ortho.cu")).read()
    raw8 = text[text.index("struct Raw8"):text.index("void norm_part")]
    assert "ld.global" in raw8 and not READ_ONLY.search(raw8)
