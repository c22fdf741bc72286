"""The register split of the decode kernel cannot deadlock.

setmaxnreg takes registers from a pool that starts with what the launch left over (nothing) and
waits, without a limit, until the pool holds enough.  The control warps give registers up and the
softmax warps take them; later both return to the launch budget.  The model below takes the order
of these steps from the kernel's source and walks through every interleaving of the warps: from
each state that can be reached, all must be able to finish."""
import os
import re

from long_context_attention_fwd_b200 import build


def steps_of(text, regs):
    """[('to', registers) | ('barrier',)] in the order of the source."""
    out = []
    for m in re.finditer(r"reg_(?:de)?alloc<(\w+)>\(\)|regs_returned\(\)", text):
        out.append(("to", regs[m.group(1)]) if m.group(1) else ("barrier",))
    return out


def can_finish(launch, roles):
    """roles: [(warps, steps)].  True if no interleaving gets stuck."""
    progs = [steps for n, steps in roles for _ in range(n)]
    kinds = [i for i, (n, _) in enumerate(roles) for _ in range(n)]

    def canon(pcs):
        return tuple(sorted(zip(kinds, pcs)))

    def held(kind, pc):
        regs = launch
        for s in roles[kind][1][:pc]:
            regs = s[1] if s[0] == "to" else regs
        return regs

    start = canon([0] * len(progs))
    seen, todo = {start}, [start]
    while todo:
        state = todo.pop()
        free = sum(launch - held(k, pc) for k, pc in state)
        nexts = []
        waiting = [(k, pc) for k, pc in state if pc < len(roles[k][1]) and roles[k][1][pc][0] == "barrier"]
        if len(waiting) == len(state):
            nexts.append(tuple(sorted((k, pc + 1) for k, pc in state)))
        for i, (k, pc) in enumerate(state):
            if pc == len(roles[k][1]) or roles[k][1][pc][0] == "barrier":
                continue
            if roles[k][1][pc][1] - held(k, pc) <= free:
                nexts.append(tuple(sorted(state[:i] + ((k, pc + 1),) + state[i + 1:])))
        if not nexts and any(pc < len(roles[k][1]) for k, pc in state):
            return False
        for x in nexts:
            if x not in seen:
                seen.add(x)
                todo.append(x)
    return True


def test_the_model_sees_the_deadlock():
    """Control warps that take their registers back without waiting can starve the softmax warps."""
    control = [("to", 72), ("to", 168)]
    softmax = [("to", 216), ("to", 168)]
    assert not can_finish(168, [(4, control), (8, softmax)])
    assert can_finish(168, [(4, control[:1] + [("barrier",)] + control[1:]), (8, softmax + [("barrier",)])])


def test_decode_kernel_register_split_cannot_deadlock():
    text = open(os.path.join(build.CSRC, "attn_decode.cuh")).read()
    regs = {n: int(v) for n, v in re.findall(r"constexpr int (kRegs\w+) = (\d+);", text)}
    body = text[text.index("  if (warp >= 8) {"):text.index("  // ---- teardown")]
    cut = body.index("  } else {\n    reg_alloc<kRegsCompute>")
    control, softmax = steps_of(body[:cut], regs), steps_of(body[cut:], regs)
    assert ("to", regs["kRegsControl"]) in control and ("to", regs["kRegsCompute"]) in softmax
    assert can_finish(regs["kRegsLaunch"], [(4, control), (8, softmax)])
