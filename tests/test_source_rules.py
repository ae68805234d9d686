"""Rules of the kernel sources that neither the compiler nor a GPU run can be
relied on to catch, checked on the CPU by reading the sources.

tcgen05.ld (tmem_load_32cols) leaves its destination registers undefined
until tcgen05.wait::ld (tmem_load_wait) has completed. The wait is a volatile
asm with a memory clobber: it keeps memory accesses after it, but not
arithmetic on the loaded registers, which the compiler may schedule above it
(an alpha * acc computed that early reads whatever the registers held before
the load landed). Every register array a TMEM load writes must therefore
pass through tmem_regs_ready, which reads and rewrites them, after the wait
and before anything else is loaded or waited for.
"""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "dense_fp32_gemm_major_gb300", "csrc")

_EVENT = re.compile(r"tmem_load_(?:16|32)cols\([^;]*?,\s*(?P<ld>\w+)\)\s*;"
                    r"|(?P<wait>tmem_load_wait\(\)\s*;)"
                    r"|tmem_regs_ready\((?P<ready>\w+)\)\s*;")


def _strip_comments(text: str) -> str:
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


def fence_violations(text: str):
    """(line, message) for each TMEM load whose registers are not fenced after
    the wait that follows it."""
    text = _strip_comments(text)
    out = []
    loaded, waited = set(), set()
    for m in _EVENT.finditer(text):
        line = text.count("\n", 0, m.start()) + 1
        if m.group("ld"):
            if waited:
                out.append((line, f"load before {sorted(waited)} passed tmem_regs_ready"))
                waited = set()
            loaded.add(m.group("ld"))
        elif m.group("wait"):
            if waited:
                out.append((line, f"second wait before {sorted(waited)} passed tmem_regs_ready"))
            waited, loaded = set(loaded), set()
        else:
            name = m.group("ready")
            if name not in waited:
                out.append((line, f"tmem_regs_ready({name}) without a pending waited load"))
            waited.discard(name)
    if loaded:
        out.append((0, f"loads of {sorted(loaded)} never waited for"))
    if waited:
        out.append((0, f"{sorted(waited)} never passed tmem_regs_ready"))
    return out


def test_every_tmem_load_is_fenced_after_its_wait():
    checked = 0
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith((".cu", ".cuh")) or name == "ptx.cuh":
            continue
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        checked += len(re.findall(r"tmem_load_wait\(\)\s*;", text))
        bad = fence_violations(text)
        assert not bad, f"{name}: {bad}"
    assert checked >= 4  # the epilogue's four paths


def test_rule_catches_an_unfenced_use():
    # the rule itself, on made-up code: a wait with no fence, a fence of the
    # wrong array, and the correct form
    bad = """
      tmem_load_32cols(t, r0);
      tmem_load_32cols(t + 32, r1);
      tmem_load_wait();
      tmem_regs_ready(r0);
      float x = p.alpha * __uint_as_float(r1[0]);
    """
    assert fence_violations(bad), "missing fence of r1 not reported"
    wrong = """
      tmem_load_32cols(t, r);
      tmem_load_wait();
      tmem_regs_ready(q);
    """
    assert fence_violations(wrong)
    good = """
      tmem_load_32cols(t, r0);
      tmem_load_32cols(t + 32, r1);
      tmem_load_wait();
      tmem_regs_ready(r0);
      tmem_regs_ready(r1);
      tmem_load_32cols(t + 64, r0);
      tmem_load_wait();  // comment
      tmem_regs_ready(r0);
    """
    assert fence_violations(good) == []


# A kernel that starts before the launch ahead of it has ended (griddepcontrol.wait)
# waits for that end on every way out: the launch behind it waits for this one's end
# alone, and builds on both.

_WAIT = r"(?:grid_dependency_wait\(\)|asm volatile\(\"griddepcontrol\.wait;\"[^;]*)\s*;"


def _kernels(text):
    """(name, body) of each __global__ function."""
    for m in re.finditer(r"__global__\s+void\s", text):
        bounds = re.compile(r"(?:__launch_bounds__\((?:[^()]|\([^()]*\))*\)\s*)?").match(text, m.end())
        head = re.compile(r"(\w+)\s*\(").search(text, bounds.end())
        at = end = text.index("{", head.end())
        depth = 0
        while True:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
            if depth == 0:
                break
        yield head.group(1), text[at:end]


def _block_before(body, at):
    """(depth, text before `at` in the block around it, blocks in it left out)"""
    depth = [""]
    for c in body[:at]:
        if c == "{":
            depth.append("")
        elif c == "}":
            depth.pop()
            depth[-1] += "}"
        else:
            depth[-1] += c
    return len(depth) - 1, depth[-1]


def early_returns(text):
    """Kernels of the source with a wait, and what returns without one."""
    bad, kernels = [], []
    for name, body in _kernels(_strip_comments(text)):
        if not re.search(_WAIT, body):
            continue
        kernels.append(name)
        top = [w.end() for w in re.finditer(r"(?<=[;{}])\s*" + _WAIT, body)
               if _block_before(body, w.end())[0] == 1]  # (behind no condition)
        for m in re.finditer(r"\breturn\s*;", body):
            depth, before = _block_before(body, m.start())
            if not any(w < m.start() for w in top) and not (depth > 1 and re.search(_WAIT, before)):
                bad.append(name)
    return kernels, bad


def test_dependent_launches_wait_before_they_return():
    kernels = []
    for name in sorted(os.listdir(CSRC)):
        if name.endswith(".cu"):
            with open(os.path.join(CSRC, name)) as f:
                found, bad = early_returns(f.read())
            assert not bad, f"{name}: {bad}"
            kernels += found
    assert {"w4_kernel", "seg_tc_kernel", "route_kernel", "scale_kernel"} <= set(kernels)


def test_rule_catches_a_return_without_a_wait():
    kernel = """
template <int V> __global__ void __launch_bounds__(f(V), 2) a_kernel(const P p) {
  if (p.n == 0) { %s return; }
  if (p.ahead) { grid_dependency_wait(); }
  if (!p.ahead) grid_dependency_wait();
  if (p.m == 0) %s
}"""
    assert early_returns(kernel % ("", "")) == (["a_kernel"], ["a_kernel"])
    assert early_returns(kernel % ("grid_dependency_wait();", ";")) == (["a_kernel"], [])
    assert early_returns(kernel % ("grid_dependency_wait();", "return;")) == (["a_kernel"], ["a_kernel"])


# The checked build looks at every index that a kernel computes: what the router's and
# the rows' kernels read and write beside their matrices stands behind index_ok, in the
# same statement or in the condition around it.

def unchecked_accesses(text):
    bad = []
    for m in re.finditer(r"p\.(?:mask|bias|weights|dweights|experts|order|places|hist|partials)\s*(?:\[|\+ )",
                         _strip_comments(text)):
        before = _strip_comments(text)[max(0, m.start() - 240):m.start()]
        block = before[before.rfind("}") + 1:]
        if "index_ok(" not in block:
            bad.append(m.group())
    return bad


def test_accesses_beside_the_matrices_are_checked():
    for name in ("route.cu", "route_rows.cu", "clip.cu"):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        assert unchecked_accesses(text) == [], name
    assert unchecked_accesses("if (a) { f(); }\n const float w = p.weights[s];") == ["p.weights["]
    assert unchecked_accesses("if (index_ok(1, s, 1, n)) { p.experts[s] = e; p.weights[s] = w; }") == []
