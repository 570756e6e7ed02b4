"""After a wait inside a kernel ran out, its CTA's other waits pass and what they
guarded may change while it is read.  The warps still have to meet: read from
the sources, no barrier stands under a condition that could then differ between
the warps or lanes that it joins (no GPU needed)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gradient_allreduce_homomorphic_gb300",
                    "csrc")


def kernel(name, head):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    begin = text.index("{", text.index(head))
    depth, at = 1, begin + 1
    while depth:
        depth += {"{": 1, "}": -1}.get(text[at], 0)
        at += 1
    return text[begin + 1:at - 1]


def conditions(body, at):
    """The heads of the blocks around a place: what stands between each one's brace and the statement before it."""
    heads, depth = [], 0
    for i in range(at - 1, -1, -1):
        if body[i] == "}":
            depth += 1
        elif body[i] == "{":
            if depth:
                depth -= 1
            else:
                start = max(body.rfind(c, 0, i) for c in ";{}") + 1
                heads.append(body[start:i].strip())
    return heads


def test_named_barriers_of_the_distillation():
    body = kernel("distill.cu", "distill_stream_kernel(")
    groups = [m.start() for m in re.finditer(r"\bbar_group<", body)]
    assert len(groups) == 2
    for at in groups:
        assert not any("live" in head for head in conditions(body, at)), conditions(body, at)
        skipped = body[:at]
        loop = max(skipped.rfind("for (uint32_t u"), skipped.rfind("for (int64_t row"))
        assert not re.search(r"\blive\)\s*continue", skipped[loop:])


def test_shared_flags_are_read_once_for_a_warp():
    body = kernel("distill.cu", "distill_stream_kernel(")
    reads = re.findall(r"[^\n]*\b(?:h|header\[e\])\.live\b(?!\s*=[^=])[^\n]*", body)
    assert len(reads) == 2 and all("__any_sync(0xFFFFFFFFu," in line for line in reads), reads


def test_no_cta_of_a_cluster_leaves_before_its_pairs_have_come():
    """A wait that ran out skips the second group's waits for them: behind the cluster barrier they are waited for with a
    limit of their own."""
    body = kernel("distill.cu", "distill_stream_kernel(")
    assert "st.async" in body
    end = body[body.rindex("__syncthreads();"):]
    assert end.index("cluster_barrier();") < end.index("failed)") < end.index("int given_up = 0;") < end.index("mbar_wait(met + 8 * at,")
    assert "&given_up" in end
