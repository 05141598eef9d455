"""Properties of the 4-bit attention kernel that no run shows without an expired wait or a foreign kernel before it, read
from its source: what its roles do after a wait that failed, and what it takes before the stream's earlier work is done."""
import os
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_indexer_e4m3_gb300", "csrc",
                   "attn_kv4_kernel.cuh")
HARDWARE = ("named_bar_sync(", "bar_or(", "__syncthreads(", "cluster_sync", "bar.sync")  # barriers whose wait has no limit


@pytest.fixture(scope="module")
def code():
    text = re.sub(r"//[^\n]*", "", open(SRC).read())
    return text[text.index("sparse_attn_kv4_kernel("):]


@pytest.fixture(scope="module")
def roles(code):
    marks = ["const auto bring_q", "if (warp >= kKv4FirstConv) {", "} else if (warp >= 4) {", "} else if (warp >= 1) {",
             "const uint32_t on = elect_one();", "if (kSingle && shares > 1) {\n"]
    at = [code.index(m) for m in marks[:-1]]
    at.append(code.index(marks[-1], at[-1]))
    assert at == sorted(at)
    return dict(zip(["bring_q", "convert", "softmax", "scout", "issue"], (code[a:b] for a, b in zip(at, at[1:]))))


def test_roles_wait_with_a_limit(roles):
    for name in ("bring_q", "convert", "scout", "issue"):
        for barrier in HARDWARE:
            assert barrier not in roles[name], (name, barrier)


def test_softmax_warps_pass_the_same_hardware_barriers(roles):
    """They enter a unit together (a vote over all of them that sees the abort flag); inside its blocks they meet at a hardware
    barrier in the first only, which none may leave, and all leave a unit at its end."""
    text = roles["softmax"]
    enter = text.index("if (bar_or(kTcEpiBar, kKv4SoftThreads, *abort_flag != 0)) break;")
    blocks = text.index("for (int b = 0; b < nb; ++b, ++gb) {")
    end = text.index("float l[kKv4SoftHeads];")
    assert text.index("const int nb = misc[n & 1];") < enter < blocks < end
    assert not any(h in text[enter + 10:end] for h in HARDWARE)
    assert re.findall(r"meet\(([^)]*)\)", text[blocks:end]) == ["b == 0"] * 2
    leave = re.findall(r"if \(([^\n]*)\) (?:break|return|continue);", text[blocks:end])
    assert leave == ["b % kLook == kLook - 1 && gone()", "b > 0 && gone()"]
    assert "break" not in text[end:] and "return" not in re.sub(r"\[[^\]]*\]\([^)]*\) \{ return [^}]*\}", "", text[end:])


def test_decisions_are_the_warp_s(roles):
    """What a warp's lanes read after a wait that may have failed for some of them and decide by, they vote on."""
    text = roles["softmax"]
    for name in ("raise = __any_sync(0xffffffffu, misc[16 + checks % 3] != 0)", "far = __any_sync(0xffffffffu, apart)",
                 "if (__any_sync(0xffffffffu, qfac[lane] != kQFac || qfac[32 + lane] != kQFac))"):
        assert name in text, name
    for use in re.finditer(r"if \(apart\)|if \(valid\)|if \(rs", text):
        raise AssertionError(use.group())


def test_block_counts_are_used_after_success_only(roles):
    text = roles["convert"]
    body = text[text.index("const auto take_unit"):]
    assert body.index("mbar_wait(&unit_full") < body.index("if (gone()) return -1;") < body.index("nb = misc[n & 1]")
    assert "if (nb < 0) break;" in body
    text = roles["scout"]
    for wait, use in (("mbar_wait(&unit_empty", "misc[n & 1] = nb"), ("mbar_wait(&ent_empty", "ent_s[slot * kTcAttnKeys + 32 * i + lane] =")):
        a, b = text.index(wait), text.index(use)
        assert "if (gone()) break;" in text[a:b]


def test_issue_role_checks_every_wait(roles):
    text = roles["issue"]
    text = text[text.index("const auto score"):]
    calls = [m.start() for m in re.finditer(r"(?<![\w_])wait\(", text)]
    assert len(calls) >= 5 and all(text[at - 1] == "!" for at in calls)


def test_start_values(code):
    """Counts, flags and page ids are defined before any role reads them."""
    setup = code[:code.index("__syncthreads()")]
    assert "misc[threadIdx.x] = 0" in setup and "ent_s[i] = make_int2(-1, 0)" in setup


def test_tensor_memory_is_taken_behind_the_stream(code):
    """A kernel that lets its dependents start early may allocate tensor memory after that: one of them that holds all of an
    SM's and waits for that kernel would never be done."""
    assert code.index("wait_stream();") < code.index("tmem_alloc(")
