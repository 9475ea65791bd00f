"""What the e4m3 kernels do ahead of pdl_wait(), where the kernel before still runs, by what is allowed rather than by what is not: barriers,
addresses and notes to the caches. And where their waits are. Each check is tried on sources with a mistake in them."""

import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_group_quantized_gb300", "csrc")
KERNELS = ("f8_quant.cu", "f8_few.cu", "f8_mid.cu", "f8_many.cu")

CALLS = {"if", "for", "volatile", "__align__", "__syncwarp", "tc_smem", "tc_mbar_init", "tc_fence_proxy", "f8_map_ahead", "f8_rank", "f8_blocks",
         "mid_block", "few_ahead"}
INSTRUCTIONS = ("prefetch.global.L2 ", "fence.mbarrier_init.release.cluster;", "barrier.cluster.arrive.release.aligned;")
SHARED = {"part", "most", "smem_raw", "bars", "full", "empty", "sf_full", "sf_free", "acc_full"}  # shared memory of the CTA
ARGUMENTS = {"p.w", "p.w_stride"}  # pointers and strides among the arguments themselves


def source(name):
    return re.sub(r"//.*", "", open(os.path.join(CSRC, name), encoding="utf-8").read())


def ahead(text):
    """What stands ahead of the wait in each kernel of a source."""
    kernels = re.split(r"__global__", text)[1:]
    assert kernels
    return [k[k.index("{") + 1:k.index("pdl_wait();")] for k in kernels]


def not_allowed(body):
    """What in it is none of the things that a kernel may do ahead of its wait."""
    out = [s for s in re.findall(r'"([^"]*)"', body) if not s.startswith(INSTRUCTIONS) and s not in ("l", "memory")]
    body = re.sub(r'"[^"]*"', "", body)
    out += [c for c in re.findall(r"(\w+)\s*(?:<[^;(){}]*>)?\s*\(", body) if c not in CALLS]
    body = re.sub(r"__shared__[^;]*;", ";", body)
    out += [s for s in re.findall(r"([\w.>\]-]+?)\s*\[", body) if s not in SHARED | ARGUMENTS]
    out += re.findall(r"\]\s*\[", body) + re.findall(r"->", body)
    # a star that neither declares a pointer nor multiplies
    body = re.sub(r"\b(?:uint64_t|unsigned char|volatile int)\s*\*\s*\w+ =[^;]*;", lambda m: re.sub(r"\*\s*(?=\w+ =)", "", m.group(0)), body)
    out += re.findall(r"(?:^|[=(,;{}&|?:<>+\-!]|\breturn)\s*\*\s*[\w(]", body)
    return out


@pytest.mark.parametrize("name", KERNELS)
def test_ahead_of_the_wait(name):
    for body in ahead(source(name)):
        assert not not_allowed(body), name


MISTAKES = ["const int e = p.xs[0];", "uint4 v = f8_ld_weights(p.w[0]);", "const uint4 v = f8_ld_weights(p.w[0] + 16 * lane);", "int e = p.w[0][3];",
            "int e = p.ws[0][0];", "const int e = *p.x;", "int e = *(const int*)p.x;", "int e = 1 + *p.x;", "f(*p.x);", "uint4 v = *reinterpret_cast<const uint4*>(p.x);",
            "norm_load<F32>(n, row, 0, raw);", "const float f = n.h[0];", "const int e = scale[3];", "int e = x[threadIdx.x];", "f8_load<1>(stages, &mx, 0, 0, 0);",
            "tmem_alloc(&s_tmem, 512);", "f8_tmem_alloc<2>(&s_tmem, 512);", 'asm volatile("ld.global.u32 %0, [%1];" : "=r"(e) : "l"(p.x));',
            "const int e = p.ctrl->status;", "p.y[0] = 0;", "*p.y = 0;", "if (*p.x) return;", "load(cur);"]


@pytest.mark.parametrize("name", KERNELS)
def test_a_read_ahead_of_the_wait_is_found(name):
    text = source(name)
    for mistake in MISTAKES:
        wrong = text.replace("pdl_wait();", mistake + " pdl_wait();")
        assert all(not_allowed(body) for body in ahead(wrong)), (name, mistake)


def waits(texts):
    """Loops that test a barrier, by source; waits written by hand; and what is wrong with them."""
    loops, wrong = [], []
    for name, text in texts.items():
        wrong += [name + ": " + s for s in re.findall(r"mbarrier\.(?:try|test)_wait", text) if name != "tc.cuh"]
        for m in re.finditer(r"\btc_mbar_(?:try|try_suspend|wait)\(", text):
            start = text.rfind("\n", 0, m.start()) + 1
            line = text[start:text.index("\n", m.start())]
            if re.match(r"\s*while \(!tc_mbar_try_suspend\(m, parity\)\) \{", line):
                body = text[m.start():text.index("\n  }", m.start())]
                loops.append(body)
                if not re.search(r"tc_time\(\) - t0\) > kF8TimeoutNs \|\| \+\+it > \(1ll << 28\)", body) or "return false" not in body:
                    wrong.append(name + ": a loop without an end")
            elif "return tc_mbar_try(m, parity) || f8_wait_loop(m, parity, fail);" not in line:
                wrong.append(name + ": " + line.strip())
    if len(loops) != 1:
        wrong.append("%d loops" % len(loops))
    return wrong


def test_every_wait_goes_by_the_bounded_one():
    texts = {name: source(name) for name in KERNELS + ("f8.h", "f8_tc.cuh")}
    assert not waits(texts)
    for name, old, new in [("f8_mid.cu", "f8_wait(&done, 0, fail)", "tc_mbar_try(&done, 0)"), ("f8_tc.cuh", "> kF8TimeoutNs", "> kNever"),
                           ("f8_many.cu", "f8_wait(&empty[s], par, fail)", "tc_mbar_wait(&empty[s], par, 1ll << 62)"),
                           ("f8_tc.cuh", "while (!tc_mbar_try_suspend(m, parity)) {", "while (!g(m, parity)) {")]:
        assert old in texts[name]
        assert waits({**texts, name: texts[name].replace(old, new)}), (name, new)
