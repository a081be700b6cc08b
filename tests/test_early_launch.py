"""Kernels that launch_early starts, read in the sources: an access before the wait for the kernel in
front is wrong in no run, or in one of many, so it is looked for where it is written."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "routing_dispatch_expert_router_gb300", "csrc")


def bodies():
    """(kernel's name, its text from the parameters to the end) of every kernel that launch_early
    starts; what follows a brace in the first column is not the kernel's."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        with open(path) as f:
            text = f.read()
        launched = "\n".join(text[m.start():m.start() + 160] for m in re.finditer(r"launch_early\(", text))
        launched += "\n".join(re.findall(r"auto kern = .*?;", text, re.S)) if "launch_early(kern" in text else ""
        for m in re.finditer(r"__global__ void\b.*?\b(\w+_kernel)\(", text, re.S):
            if m.group(1) in launched:
                body = text[m.end():]
                yield m.group(1), re.sub(r"//.*", "", body[:body.index("\n}\n")])


def test_every_thread_waits_before_its_first_access_to_memory():
    seen = []
    for name, body in bodies():
        params, code = body[:body.index(") {")], body[body.index(") {"):]
        waits = [m.start() for m in re.finditer(r"grid_dependency_wait\(\)", code)]
        assert len(waits) == 1, (name, "one wait, for all threads")
        before = code[:waits[0]]
        line = before[before.rindex("\n"):]
        assert re.fullmatch(r"\n  ptx::", line), (name, "at the kernel's own level: no branch around it")
        assert "return;" not in before and "launch_dependents" not in before, name
        # pointers among the parameters, and those in a parameter structure
        for pointer in re.findall(r"\*\s*(?:__restrict__\s+)?(\w+)", params):
            assert not re.search(r"(?<![\w.])%s\b" % pointer, before), (name, pointer)
        for access in (r"\bp\.\w+\s*\[", r"__ld\w+\(", r"\bld\w*_v4\(", r"record_status", r"cp_async\d", r"tma_load", r"\batomic"):
            assert not re.search(access, before), (name, access)
        seen.append(name)
    assert {"permute_hist_kernel", "permute_rank_kernel", "permute_scatter8_kernel", "rmsnorm_fwd_kernel",
            "rmsnorm_fwd_ring_kernel", "rmsnorm_bwd_kernel", "dgamma_kernel", "product_few_kernel",
            "product_short_kernel", "ragged_pair_kernel"} <= set(seen)
