"""The cluster merge of the 4-bit attention: no CTA leaves while a copy to or from it is in flight, not even
after a wait that ran out.

The protocol is read from the kernel's source, in its order: PUSH (bulk copies of partials to every CTA),
RECEIVE (the bounded wait for one's own), ARRIVE and AWAIT of the cluster barrier, and the exit.  All
interleavings of two CTAs are walked.  A copy lands at any time after it is issued; a RECEIVE that starts
when all copies to its CTA have been issued ends with them, any other may run out first."""
import os
import re

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_decoding_verify_step_gb300", "csrc",
                   "kv4_attention.cu")
OPS = {"bulk_push": "PUSH", "mbar_wait": "RECEIVE", "cluster_arrive": "ARRIVE", "cluster_arrive_relaxed": "ARRIVE", "cluster_wait": "AWAIT"}


def protocol():
    """[(op, only after a RECEIVE that ran out)] of a CTA of a cluster of two or more."""
    text = re.sub(r"//[^\n]*", "", open(SRC).read())
    kernel = text[text.index("kv4_attention_kernel("):text.index("kv4_merge_kernel(")]
    first = kernel.index("cluster_arrive()")
    merge = kernel[kernel.index("if constexpr (CL)", first):]
    merge = merge[:merge.index("return;")]
    ops = [("ARRIVE", False)]
    for hit in re.finditer(r"(if \(!ok\)[^;{]*?)?\b(bulk_push|mbar_wait|cluster_arrive_relaxed|cluster_arrive|cluster_wait)\(", merge):
        ops.append((OPS[hit.group(2)], bool(hit.group(1))))
    return ops


def unsafe_exit(ops):
    """Whether some interleaving lets a CTA leave with a copy in flight to or from it."""
    # per CTA: place, may its running RECEIVE run out (None: none running), did one run out, barrier arrivals;
    # copies (from, to): 0 not issued, 1 in flight, 2 landed
    start = (tuple((0, None, False, 0) for _ in range(2)), (0, 0))
    seen, todo = {start}, [start]
    while todo:
        ctas, copies = todo.pop()
        after = []
        for i in range(2):                                   # copy i is CTA i's to the other
            if copies[i] == 1:
                after.append((ctas, tuple(2 if j == i else x for j, x in enumerate(copies))))
        for i in range(2):
            place, running, ran_out, arrived = ctas[i]
            if place == len(ops):
                if 1 in copies:
                    return True
                continue

            def put(state, new_copies=copies, i=i):
                after.append((tuple(state if j == i else s for j, s in enumerate(ctas)), new_copies))

            op, conditional = ops[place]
            if conditional and not ran_out:
                put((place + 1, None, ran_out, arrived))
            elif op == "PUSH":
                put((place + 1, None, ran_out, arrived), tuple(1 if j == i else x for j, x in enumerate(copies)))
            elif op == "ARRIVE":
                put((place + 1, None, ran_out, arrived + 1))
            elif op == "AWAIT":
                if ctas[1 - i][3] >= arrived:
                    put((place + 1, None, ran_out, arrived))
            elif running is None:
                put((place, copies[1 - i] == 0, ran_out, arrived))
            else:
                if copies[1 - i] == 2:
                    put((place + 1, None, ran_out, arrived))
                if running:
                    put((place + 1, None, True, arrived))
        for s in after:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return False


def test_the_walk_finds_what_it_looks_for():
    done = [("ARRIVE", False), ("AWAIT", False), ("PUSH", False), ("RECEIVE", False)]
    assert unsafe_exit(done)                                                   # leaves with its own copy in flight
    assert unsafe_exit(done + [("ARRIVE", False), ("AWAIT", False)])           # the other's push may come after
    assert not unsafe_exit([("ARRIVE", False), ("AWAIT", False)])


def test_no_cta_leaves_a_cluster_with_a_copy_in_flight():
    ops = protocol()
    assert [o for o, _ in ops].count("PUSH") == 1 and ops[0] == ("ARRIVE", False)
    assert [o for o, c in ops if not c].count("ARRIVE") == [o for o, c in ops if not c].count("AWAIT")
    assert not unsafe_exit(ops)
