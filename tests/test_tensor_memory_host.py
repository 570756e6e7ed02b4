"""Tensor memory is allocated, shared and given back as its rules ask, read from
the sources (no GPU needed)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gradient_allreduce_homomorphic_gb300",
                    "csrc")


def source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def body(text, head):
    """The braces that follow `head`, their contents."""
    begin = text.index("{", text.index(head))
    depth, at = 1, begin + 1
    while depth:
        depth += {"{": 1, "}": -1}.get(text[at], 0)
        at += 1
    return text[begin + 1:at - 1]


def test_permit_to_allocate_is_given_back_at_once():
    """CTAs that share an SM allocate one after another: none waits for another's end."""
    text = source("tensorcore.cuh")
    order = re.findall(r"tcgen05\.(alloc|relinquish_alloc_permit)\.(cta_group::\d)", body(text, "void tmem_alloc("))
    assert order == [(op, g) for g in ("cta_group::1", "cta_group::2") for op in ("alloc", "relinquish_alloc_permit")]
    assert "relinquish" not in body(text, "void tmem_free(")


def test_tensor_memory_is_given_back_after_the_products():
    """Also where a wait ran out and lets all others pass: the warp that sends off products ends with a commit behind
    them and a wait of its own limit for it, and the warp that copies scales with a wait for its copies."""
    text = source("matmul.cu")
    for head in ("matmul_kernel(", "matmul_pair_kernel("):
        kernel = body(text, head)
        warps = re.split(r"if \(warp == (\d)[^)]*\) \{", kernel)
        roles = dict(zip(warps[1::2], warps[2::2]))
        assert re.search(r"tc_commit<\d>\(done\);\s*__syncwarp\(\);\s*products_done\(done\);\s*\} else $", roles["1"]), head
        assert re.search(r"copy_async_wait\(\);\s*\}", roles["2"]), head
    wait = body(text, "void products_done(")
    assert "int given_up = 0;" in wait and "failed" not in wait
