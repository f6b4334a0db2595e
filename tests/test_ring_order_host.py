"""Order of reads and refills of shared memory that asynchronous copies write, as the sources have it.

A copy by TMA or cp.async.bulk belongs to another proxy than a thread's loads.  A slot that is handed back right behind
loads can be refilled while they are still on their way to registers, at full speed and now and then, so no run shows
that it cannot happen: the order has to be there in the source.  It is there where a proxy fence stands between the loads
and the arrival, or an instruction that cannot start before the loaded values are there."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_expert_ffn_dispatch_gb300", "csrc")
FENCE = r"fence_proxy_async_smem\(\);"


def source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def last(patterns, text):
    """Which of the patterns has the last match in the text."""
    at = {p: max([m.start() for m in re.finditer(p, text)], default=-1) for p in patterns}
    best = max(at, key=at.get)
    assert at[best] >= 0, patterns
    return best


def test_the_dp4a_ring_hands_slots_and_token_rows_back_behind_a_proxy_fence():
    src = source("moe_gemm.cu")
    loads = r"stage_dot_m<\w+>\(m, Ws"
    for arrival in (r"mbar_arrive\(&empty\[s\]\)", r"mbar_arrive\(tok_empty\)"):
        found = list(re.finditer(arrival, src))
        assert found
        for m in found:
            assert last((loads, FENCE), src[:m.start()]) == FENCE, arrival


def test_converted_codes_are_in_registers_before_their_slot_goes_back():
    """In the two kernels that widen codes into tensor memory: the stores of the converted codes come first, or a fence."""
    loads, stores = r"c\[j\] = \*reinterpret_cast", r"tmem_st32\("
    src = source("tc_gemm.cu")
    found = list(re.finditer(r"mbar_arrive\(&a8_empty", src))
    assert len(found) == 2
    for m in found:
        assert last((loads, FENCE, stores), src[:m.start()]) != loads
    src = source("w8_linear_tc.cu")
    found = list(re.finditer(r"[^=] hand_back\(\);", src))
    assert len(found) == 2
    for m in found:
        assert last((loads, FENCE, stores), src[:m.start()]) != loads


def test_the_one_launch_scratch_is_done_with_before_token_rows_are_copied_over_it():
    """The dispatch's scratch is written and read by threads, in the area that bulk copies of token rows take after the
    `ready` barrier: the producer, past that barrier, fences before its first copy."""
    src = source("moe_gemm.cu")
    wait = src[src.index("auto wait_ready = [&]"):]
    wait = wait[:wait.index("};")]
    seen = wait.index("ss.ready_seen = true;")
    assert wait.index("mbar_wait_bounded(ready") < seen and re.search(FENCE, wait[seen:])


def test_what_the_ctas_of_a_pair_tell_each_other_has_the_clusters_scope():
    """An arrival at the other CTA's barrier, or a wait for one, whose scope is not named has the CTA's own and orders
    nothing between the two."""
    src = source("w8_linear_tc.cu") + source("device_prims.cuh")
    arrivals = re.findall(r'"mbarrier\.arrive[\w.:]*\.shared::cluster[^"]*"', src)
    assert arrivals and all(re.match(r'"mbarrier\.arrive\.(relaxed|release)\.cluster\.', a) for a in arrivals), arrivals
    assert "mbarrier.try_wait.parity.acquire.cluster" in src


def test_both_ctas_token_copies_complete_the_barrier_that_the_products_wait_for():
    """Handed on by a thread of the second CTA, they would need its release over the cluster."""
    src = source("w8_linear_tc.cu")
    landed = re.search(r"landed = FORM == kTwo \? remote_of\(&bar\.full\[s\], 0\)", src)
    copies = re.findall(r"\bpair_tma_load_2d\(to[^;]*;", src)
    assert landed and len(copies) == 2 and all(c.endswith("landed);") for c in copies)
    assert re.search(r"if \(!side_of_pair\) moe::mbar_arrive_expect_tx\(&bar\.full\[s\], bytes\)", src)


def test_kernels_that_hand_registers_on_are_launched_only_with_what_the_split_needs():
    """setmaxnreg.inc waits until the block has the registers: built with fewer a thread than the split adds up to, it would
    wait for ever.  Each such kernel's launch names the number that its static_assert counts with."""
    users = [f for f in sorted(os.listdir(CSRC)) if "setmaxnreg.inc" in source(f)]
    assert users == ["kv_attention_chunk.cu", "w8_linear_tc.cu"]
    for f in users:
        src = source(f)
        assert re.search(r"static_assert\([^;]*<= kThreads \* kLaunchRegs", src)
        assert re.search(r"allow_smem\(k, kMaxSmem, allowed, [^;]*kLaunchRegs", src)
    ops = source("layer_ops.cuh")
    assert re.search(r"if \(is\.numRegs < regs\) return", ops)
