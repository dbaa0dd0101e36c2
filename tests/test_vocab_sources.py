"""What the vocabulary losses' source has to hold to that no run shows (no GPU: it is read as text). TMEM's loads, stores and waits
are `.sync.aligned`: all lanes of a warp execute them together, so a branch that lanes take differently has to have ended, by a
warp-wide operation, before the next of them."""
import re

import pytest

from tests.test_training_loads import body

EVENTS = re.compile(r"(?P<apart>row0 \+ lane < |\brow < g\.rows\b|\blane == 0\b|\blane < g\.rows\b|listed\.e < listed\.end|\bif \(mine\)|at >= 32)"
                    r"|(?P<together>__syncwarp\(\)|__all_sync\(|__any_sync\(|__shfl_sync\(|__reduce_add_sync\(|__ballot_sync\(|__syncthreads\(\)|"
                    r"acquire\(\)|release\(\))"
                    r"|(?P<tmem>tmem_(load|load16|wait|store|stored)\()|(?P<tmem2>tcgen05\.(ld|wait::ld|st|wait::st)\.sync\.aligned)")


def walk(text):
    apart = None
    for m in EVENTS.finditer(text):
        if m["apart"]:
            # (an argument of a warp-wide operation is no branch)
            before = text[max(0, m.start() - 60):m.start()]
            if re.search(r"__(any|all|ballot|reduce_add)_sync\([^;{]*$", before) or re.search(r"(const bool|\bbool) \w+ = [^;{]*$", before):
                continue
            apart = m
        elif m["together"]:
            apart = None
        else:
            assert apart is None, f"'{text[apart.start():m.end()][:300]}'"


def loop(text, head):
    """The body of the loop that starts with `head`."""
    at = text.index(head)
    at = text.index("{", at)
    end, depth = at + 1, 1
    while depth:
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        end += 1
    return text[at + 1:end - 1]


@pytest.mark.parametrize("name", ["logits_half", "keep_listed", "logits_epilogue", "grad_epilogue", "vocab_few_kernel", "vocab_few_grad_kernel",
                                  "vocab_product_kernel"])
def test_lanes_meet_before_tmem(name):
    walk(body("pg_vocab.cu", name))


def test_lanes_meet_around_the_loop_over_few_rows():
    one = loop(body("pg_vocab.cu", "vocab_few_kernel"), "for (int c0 = 0; c0 < g.rows")
    assert "tmem_load" in one and "g.sums" in one
    walk(one + one)
