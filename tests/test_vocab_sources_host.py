"""The vocabulary layer's products keep the rules of kernels whose waits are bounded,
read from the source (no GPU needed): after a wait ran out every other wait passes, and
the CTA pair still meets, waits for its copies and products, and gives its tensor memory back."""
import re

from test_bounded_waits_host import conditions, kernel

BODY = kernel("vocab.cu", "vocab_product_kernel(")


def roles():
    warps = re.split(r"if \(warp (==|>=) (\d)[^{]*\) \{", BODY[BODY.index("if (warp == 0 && lane == 0)"):])
    return {number: text for number, text in zip(warps[2::3], warps[3::3])}


def test_tensor_memory_is_given_back_after_the_products():
    """The warp that sends off products ends with a commit behind them and a wait of its own limit for it."""
    text = roles()["1"]
    end = text[text.rindex("tc_commit<2>(done);"):]
    assert re.match(r"tc_commit<2>\(done\);\s*__syncwarp\(\);\s*int given_up = 0;\s*mbar_wait\(done, 0, &given_up\);\s*\} else $", end)


def test_copies_land_before_the_pair_ends():
    """Where the issue of copies stopped, the CTA whose barriers count them waits for those under way with a limit of its own."""
    text = roles()["0"]
    assert re.search(r"if \(!ok && rank == 0\) drain_stages\(full, stages, issued, s, turn\);\s*\} else $", text)
    drain = kernel("vocab.cu", "void drain_stages(")
    assert "int given_up = 0;" in drain and "&given_up" in drain and "failed" not in drain
    # one loop iteration issues only behind a wait that was not given up, and counts what it issued
    loop = text[text.index("for (int32_t c = it.c0"):]
    assert loop.index("mbar_wait(empty + 8 * s, turn, &failed)") < loop.index("break;") < loop.index("tma_load") < loop.index("issued =")


def test_barriers_stand_under_no_condition():
    for barrier in ("__syncthreads();", "cluster_barrier();"):
        places = [m.start() for m in re.finditer(re.escape(barrier), BODY)]
        assert len(places) == 2
        for at in places:
            assert conditions(BODY, at) == [], conditions(BODY, at)
    end = BODY[BODY.rindex("__syncthreads();"):]
    assert end.index("cluster_barrier();") < end.index("GAR_STATUS_TIMEOUT") < end.index("tmem_free<2>(tmem, 512);")


def test_no_loop_ends_early_for_a_wait():
    """Products and epilogue go through all their tiles whatever their waits say: only the copies look at the answer."""
    found = roles()
    for number in ("1", "2"):
        text = re.sub(r"ready = mbar_test\([^;]*;", "", found[number])
        assert not re.search(r"(if|while|=)\s*\(?!?\s*mbar_(wait|test|try)", text), number
        assert "break;" not in text


def test_every_segment_hands_its_accumulator_back_once():
    """Each way through an epilogue's turn has one arrival for the products that wait for it: a half without columns; a
    segment of a longer sum, behind the second of its two reads; the last batch else, in either order of batches."""
    text = roles()["2"]
    arrivals = [m.start() for m in re.finditer(r"mbar_arrive_cluster\(lead_drained \+ 8 \* buf\);", text)]
    heads = [" ".join(conditions(text, at)) for at in arrivals]
    assert len(arrivals) == 4
    assert "half >= batches" in heads[0]
    assert "kForm == kLong && half < batches" in heads[1] and "u == 1" in heads[1]
    assert "kForm != kLong && u == 1 && q + 2 >= batches / 2" in heads[2]
    assert "kForm != kLong && j + 2 >= batches" in heads[3]
    for at in arrivals:  # what was read has arrived
        assert text.rindex("tc_fence_before();", 0, at) > text.rindex("tc_fence_after();", 0, at)
    for at in arrivals[1:]:
        assert text.rindex("tc_wait_ld();", 0, at) > text.rindex("tc_load32(", 0, at)
