"""What a block of the attention kernels does when a wait runs out, read from their source: it
stops where the wait is, and leaves only after every copy that it issued has landed."""
from __future__ import annotations

import re

import pytest

from tests.test_kernel_rules_host import kernels

FILES = [("attn_few.cu", "attention_few_kernel"), ("attn_tile.cu", "attention_tile_kernel")]


def statement(body: str, at: int) -> str:
    """The statement that holds `at`."""
    start = max(body.rfind(c, 0, at) for c in ";{}") + 1
    return body[start:body.index(";", at) + 1].strip()


def conditions(body: str, at: int) -> list:
    """Heads of the blocks and statements that `at` lies under, the outermost first."""
    heads, start = [], 0
    for i, ch in enumerate(body[:at]):
        if ch == "{":
            heads.append(body[start:i])
        elif ch == "}":
            heads.pop()
        if ch in ";{}":
            start = i + 1
    return [h.strip() for h in heads + [body[start:at]]]


def waits(body: str) -> list:
    """Places of the waits on a barrier of the block that end early once one has run out."""
    return [m.start() for m in re.finditer(r"\b(?:mbar_)?wait\(&sm\.", body)
            if "&never" not in statement(body, m.start())]


def loads(body: str) -> list:
    return [m.start() for m in re.finditer(r"\b(?:load_tile<|tma_load_\dd\(|bulk_load\()", body)]


@pytest.mark.parametrize("name,kernel", FILES)
def test_every_wait_is_heeded(name, kernel):
    body = kernels(name)[kernel]
    assert len(waits(body)) >= 3
    for at in waits(body):
        s, after = statement(body, at), body[body.index(";", at) + 1:]
        if re.match(r"ok = wait\(", s):                # on the spot
            assert re.match(r"\s*if \(!ok\) break;", after), s
        elif re.match(r"ptx::mbar_wait\(&sm\.s_full", s):
            assert re.match(r"\s*bool gave_up = \*abort;", after), s
        elif not re.match(r"ptx::mbar_wait\(&sm\.o_", s):   # (what follows is only read)
            assert re.match(r"ok &= wait\(|(?:if \(.*\)|else)\s+gave_up \|= !wait\(|if \(!wait\(.*break;",
                            s), s


def test_nothing_is_issued_or_released_after_a_wait_that_ran_out():
    body = kernels("attn_tile.cu")["attention_tile_kernel"]
    found = [m.start() for m in re.finditer(r"\bmma_[st]s\(|tc_commit\(&sm\.(?!done)|mbar_arrive\(&sm\.",
                                            body)]
    assert len(found) >= 10
    for at in found:
        heads = conditions(body, at)
        assert any(re.search(r"\bif \([^;]*&& (?:ok|!gave_up)\)", h) for h in heads), heads[-1]


@pytest.mark.parametrize("name,kernel", FILES)
def test_every_load_waits_for_its_stage(name, kernel):
    body = kernels(name)[kernel]
    places = loads(body)
    assert places
    for at in places:
        before = body[:at].rfind("empty")
        assert before >= 0 and re.match(r"ok = wait\(&sm\.\w*empty", statement(body, before))


@pytest.mark.parametrize("name,kernel", FILES)
def test_what_was_issued_has_landed_before_the_block_leaves(name, kernel):
    body = kernels(name)[kernel]
    last = loads(body)[-1]
    found = 0
    for m in re.finditer(r"mbar_wait\(&sm\.(\w*full)", body[last:]):
        at = last + m.start()
        if "&never" not in statement(body, at):
            continue
        found += 1
        for head in conditions(body, at):
            assert not re.search(r"\babort\b|\bif \([^)]*\bok\b", head), head
    assert found
