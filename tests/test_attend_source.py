"""What csrc/attend.cu must keep to where a run would show it only by chance: read in the source.

The kernel's cost tables lie where the loading warp later has q written by an asynchronous copy."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def source():
    with open(os.path.join(ROOT, "paged_block_sparse_vt_b200", "csrc", "attend.cu")) as f:
        text = f.read()
    return re.sub(r"//[^\n]*", "", text)


def between(text, start, end):
    i = text.index(start)
    return text[i:text.index(end, i)]


def test_no_warp_reads_the_cost_tables_while_q_may_come():
    """Behind the barrier that ends their making, the tables are read by the loading warp itself,
    and elsewhere only in blocks that end in a barrier, before any role begins."""
    body = between(source(), "attend_kernel(const AttendParams p", "struct Join")
    after = body[body.index("flag(p.status, VT_DEV_BAD_START)"):]
    roles = after[:after.index("if (warp >= kLoadWarp)")]
    reads = [m.start() for m in re.finditer(r"table[01]\b", roles)]
    assert reads
    for at in reads:
        rest = roles[at:]
        # the loading warp's own name for its line, used in its role only
        if re.match(r"table0;", rest):
            continue
        assert "__syncthreads();" in rest, roles[max(0, at - 80):at + 40]
    first = roles[:roles.index("if (SHARED && cta ==")]
    assert not re.search(r"table[01]\b", first), first
    # past the roles' start nobody but the loading warp follows that name
    loading = between(after, "if (warp == kLoadWarp)", "else if (warp == kMmaWarp)")
    uses = len(re.findall(r"\bline\[", after[after.index("if (warp >= kLoadWarp)"):]))
    assert uses == len(re.findall(r"\bline\[", loading)) > 0


def test_a_bounded_wait_has_one_answer_for_the_warp():
    """The phase is polled, and given up, by vote; and whole warps call it."""
    text = source()
    body = between(text, "bool wait(uint32_t bar", "\n}\n")
    polls = re.findall(r"(\S*\(\w*,? ?)?umma::mbar_try_wait", body)
    assert polls and all(x == "(__all_sync(kFull, " or x.endswith("__all_sync(kFull, ")
                         for x in polls), polls
    gives_up = between(body, "while (", "return false")
    assert "if (__any_sync(kFull, *abort_flag != 0 || global_ns() - t0 > kWaitNs))" in gives_up
    assert body.count("return false") == 1
    # nothing that calls it stands in a lane's own block
    for m in re.finditer(r"\bwait\(smem_u32", text):
        line = text[text.rfind("\n", 0, m.start()) + 1:m.start()]
        assert "lane" not in line, line
    for block in re.finditer(r"if \(lane == 0[^{;]*\{", text):
        depth, i = 1, block.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        assert not re.search(r"\bwait\(", text[block.end():i])


def test_every_arrival_for_the_product_warp_stands_behind_the_tensor_memory_fence():
    """A p_ready arrival lets O and S be overwritten: what its warp read from them is ordered first,
    whether or not the warp has rows of its own in this item."""
    text = source()
    arrivals = [m.start() for m in re.finditer(r"umma::mbar_arrive\(smem_u32\(&sh\.p_ready", text)]
    assert len(arrivals) == 3
    for at in arrivals:
        before = text[:at]
        # the last thing that is not an arrival, a lane's guard or a warp barrier
        block = re.sub(r"(umma::mbar_arrive\([^;]*;|if \(lane == 0\) ?\{?|__syncwarp\(\);|\s)+$", "",
                       before)
        assert block.endswith("umma::fence_before_sync();"), block[-120:]


def test_copies_and_products_in_flight_are_waited_for_whoever_gives_up():
    """The loading and the product warp may be done issuing when another warp gives up: what is in
    flight lands before the block's shared and tensor memory go, whoever gave up."""
    body = between(source(), "if (warp == kLoadWarp) {", "regs_more<kRegsSoftmax>")
    for wait_for in (r"min\(filled, \(uint32_t\)C::STAGES\)", r"sh\.q_full\), \(n_item - 1\) & 1",
                     r"umma::commit\(smem_u32\(&sh\.drain\)\)"):
        (at,) = [m.start() for m in re.finditer(wait_for, body)]
        # the open blocks around it: none of them is a condition on this warp's own giving up
        depth, i, opened = 0, at, []
        while i > 0:
            i -= 1
            if body[i] == "}":
                depth += 1
            elif body[i] == "{":
                if depth:
                    depth -= 1
                else:
                    opened.append(body[body.rfind("\n", 0, i) + 1:i].strip())
        assert opened and not any(re.search(r"\bgo\b", o) for o in opened), opened
