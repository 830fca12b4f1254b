"""What the attentions of libcosa_attn wait for once a wait has run out: read from the source, since no test makes a copy get lost."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("name,slots", [("attn_paged.cu", 3), ("attn_prefill.cu", 3)])
def test_copies_in_flight_have_one_budget_together(name, slots):
    """2 s, and 2 s more for the copies: not 2 s for each slot of the rings in turn."""
    text = open(os.path.join(ROOT, "block_sparse_long_gb300", "csrc", name)).read()
    drain = text[text.index("every copy lands before the CTA ends"):]
    drain = drain[:drain.index("__syncwarp();")]
    assert "wait_parity_bounded" not in drain
    assert len(re.findall(r"wait_until\([^;]*, since\);", drain)) == slots and drain.count("global_timer_ns()") == 1


def test_keys_count_as_in_flight_once_they_are_copied():
    """The expanded form's producer may give up between a block's keys and its values: the ring has moved past the keys by then, so
    that those waited for are the last ones of each slot."""
    text = open(os.path.join(ROOT, "block_sparse_long_gb300", "csrc", "attn_prefill.cu")).read()
    copies = text[text.index("if (keys == S::kSlots)"):text.index("every copy lands before the CTA ends")]
    assert copies.index("&krmap") < copies.index("kring.next();") < copies.index("if (values == S::kSlots)") < copies.index("vring.next();")
    drain = text[text.index("every copy lands before the CTA ends"):]
    assert "next()" not in drain[:drain.index("__syncwarp();")]


def test_the_list_of_joins_is_written_whatever_became_of_the_call():
    """A CTA that does nothing, since a wait had run out before it, leaves no entry as the workspace had it; and the join does not
    take an index that could wrap in its check."""
    text = open(os.path.join(ROOT, "block_sparse_long_gb300", "csrc", "attn_paged.cu")).read()
    joins = text[text.index("what is to be joined ===="):]
    assert "more = sm.start.any;" in joins[:joins.index("for (")]
    assert "const bool works = sm.start.any && !sm.over;" in text and "mine = works && ok;" in text
    check = text[text.index("const Join j = a.joins[blockIdx.x];"):]
    assert "static_cast<uint32_t>(j.next) + j.step * (j.parts - 2) >= 2u * kCtas" in check[:check.index("return;")]
