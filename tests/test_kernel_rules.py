"""Rules of the kernels' sources that no run on a GPU can show broken: what breaks them leaves behaviour
undefined, or shows only when a wait has run out."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_127_gb300", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))

# Warp counts that are multiples of four wherever registers are split (setmaxnreg): 4 or 8 consumers, 8 warps before the softmax.
WHOLE_GROUPS = {"C::kConsumers", "C::kSoftWarp0"}


def code_of(path):
    """A source without its comments; string literals lose their braces."""
    text = open(path).read()
    text = re.sub(r"//[^\n]*", "", text)
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.sub(r'"(?:\\.|[^"\\])*"', lambda m: m.group(0).replace("{", " ").replace("}", " "), text)


def conditions_at(code, position):
    """The conditions that the statement at `position` stands under, those of the branches before an else among them."""
    stack, chains, header_from = [], {}, 0
    for i, ch in enumerate(code[:position]):
        if ch == "{":
            header = code[header_from:i].strip()
            chain = list(chains.get(len(stack), [])) if header.startswith("else") else []
            if re.match(r"(else\s+)?if\b", header):
                chain.append(header)
            chains[len(stack)] = chain
            stack.append(chain)
            chains[len(stack)] = []
        elif ch == "}":
            stack.pop()
        if ch in "{};":
            header_from = i + 1
    return [c for chain in stack for c in chain]


def splits_a_warpgroup(condition):
    """Whether a condition on the warp's number can differ between warps 4 g .. 4 g + 3."""
    for op, bound in re.findall(r"\bwarp\s*(<=|>=|==|!=|<|>)\s*([\w:]+)", condition):
        if op not in ("<", ">="):
            return True
        if bound.isdigit():
            if int(bound) % 4:
                return True
        elif bound not in WHOLE_GROUPS:
            return True
    return False


def test_every_warp_of_a_warpgroup_runs_the_same_setmaxnreg():
    """All four warps execute the same setmaxnreg, or behaviour is undefined (and an increase may wait for good)."""
    found = 0
    for path in SOURCES:
        code = code_of(path)
        for m in re.finditer(r"setmaxnreg", code):
            found += 1
            bad = [c for c in conditions_at(code, m.start()) if splits_a_warpgroup(c)]
            assert not bad, f"{os.path.basename(path)}: setmaxnreg under {bad}"
    assert found >= 8


@pytest.mark.parametrize("condition,splits", [("if (warp < 2)", True), ("if (warp >= 4 && warp < 12)", False), ("if (warp == 0)", True),
                                              ("else if (warp < 6)", True), ("if (warp >= C::kConsumers)", False), ("if (u < MT)", False)])
def test_the_rule_tells_conditions_apart(condition, splits):
    assert splits_a_warpgroup(condition) == splits


@pytest.mark.parametrize("name", ["pa_chunk_umma.cuh", "pa_chunk_scored_umma.cuh", "pa_attend8_umma.cuh"])
def test_a_published_item_is_read_by_the_whole_warp_before_it_is_freed(name):
    """Every lane copies an item's slot, and one lane's arrive frees it: a barrier of the warp between the two."""
    code = code_of(os.path.join(CSRC, name))
    body = re.search(r"auto take = \[&\].*?\};", code, flags=re.S).group(0)
    copy, barrier = body.find("out = slot("), body.find("__syncwarp()")
    assert 0 <= copy < barrier < body.find("return got")


@pytest.mark.parametrize("name", ["pa_chunk_umma.cuh", "pa_chunk_scored_umma.cuh", "pa_attend8_umma.cuh"])
def test_softmax_warps_leave_together(name):
    """The warpgroup's barriers have no limit, so a warp that leaves the loop over items (at their end, or because its wait
    ran out) goes through one of them first: otherwise the other three might wait there for good."""
    code = re.sub(r"\s+", " ", code_of(os.path.join(CSRC, name)))
    loop = code[code.rfind("take(u,"):]           # the softmax role is the last one that takes items
    assert re.match(r"take\(u, ku?, \w+\); if \(!ok \|\| \w+\.end\) \{ (warp)?group_all\(1 \+ u, false\); break; \}", loop)
    # behind the steps: one decision for all four warps
    assert re.search(r"ok = (warp)?group_all\(1 \+ u, ok\); if \(!ok\) break;", loop)


def test_no_cache_is_read_by_the_read_only_path():
    """ld.global.nc is for memory that nothing writes while a kernel lives; a kernel launched ahead of its predecessor's
    end lives while that one writes the cache."""
    for path in SOURCES:
        assert "ld.global.nc" not in code_of(path), os.path.basename(path)
