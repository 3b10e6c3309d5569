"""The attention kernels as built, in assembly: every path from a matrix
instruction to the first other use of its result has the wait states that
gfx950 asks for, and nothing but the direct loads takes its operand from m0
(which their inline assembly writes without telling the compiler); and those
loads, whose scalar operands the compiler does not count waits for, keep the 5
wait states from a vector instruction that writes one.

Wait states: an instruction counts one, `s_nop n` counts n + 1; a vector, LDS or
memory instruction, and a matrix instruction by an operand other than the sum
that it adds to, has to keep 8 passes + 4 of them from a 32x32x16 bf16 product
whose result it reads or writes."""
import concurrent.futures
import importlib.util
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PRODUCT, NEED = "v_mfma_f32_32x32x16_bf16", 12


def builder():
    path = os.path.join(ROOT, "conv_subsampling_amd", "build.py")
    spec = importlib.util.spec_from_file_location("_dwconv_build_asm", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def registers(text):
    found = {(k, int(n)) for k, n in re.findall(r"\b([va])(\d+)\b", text)}
    for k, first, last in re.findall(r"\b([va])\[(\d+):(\d+)\]", text):
        found |= {(k, n) for n in range(int(first), int(last) + 1)}
    return found


def scalars(text):
    found = {int(n) for n in re.findall(r"\bs(\d+)\b", text)}
    for first, last in re.findall(r"\bs\[(\d+):(\d+)\]", text):
        found |= set(range(int(first), int(last) + 1))
    return found


def kernels(text):
    """Each kernel's lines: (label, None) or (name, operands)."""
    code, name = {}, None
    for line in text.splitlines():
        line = line.split(";")[0].strip()
        start = re.match(r"(_Z\w+):$", line)
        if start:
            name = start.group(1)
            code[name] = []
        elif name and re.match(r"\.L\w+:$", line):
            code[name].append((line[:-1], None))
        elif name and line and not line.startswith("."):
            parts = line.split(None, 1)
            code[name].append((parts[0], parts[1] if len(parts) > 1 else ""))
    return code


def too_early(code):
    """(matrix instruction, use, wait states between) wherever there are fewer than NEED."""
    label = {op: at for at, (op, args) in enumerate(code) if args is None}
    uses = [None if args is None else registers(args) for _, args in code]
    bad = []
    for at, (op, args) in enumerate(code):
        if not op.startswith("v_mfma"):
            continue
        assert op == PRODUCT, op
        result, todo, seen = registers(args.split(", ")[0]), [(at + 1, 0)], {}
        while todo:
            i, waited = todo.pop()
            while i < len(code) and waited < NEED and seen.get(i, NEED) > waited:
                seen[i] = waited
                name, more = code[i]
                if more is None:
                    i += 1
                    continue
                if name == PRODUCT:
                    d, a, b, c = (registers(x) for x in more.split(", ")[:4])
                    if (a | b) & result or (c & result and c != result) or (d & result and d != result):
                        bad.append((args, f"{name} {more}", waited))
                    if d == result:
                        break  # the sum goes on there
                elif uses[i] & result:
                    bad.append((args, f"{name} {more}", waited))
                    break
                if name == "s_endpgm":
                    break
                waited += int(more) + 1 if name == "s_nop" else 1
                if name == "s_branch":
                    i = label[more.strip()]
                    continue
                if name.startswith("s_cbranch"):
                    todo.append((label[more.strip()], waited))
                i += 1
    return bad


def loads_too_early(code, need=5):
    """Direct loads within `need` wait states of a vector instruction that writes one of their scalars."""
    label = {op: at for at, (op, args) in enumerate(code) if args is None}
    bad = []
    for at, (op, args) in enumerate(code):
        if args is None or not op.startswith("v_"):
            continue
        written, todo, seen = scalars(args.split(",")[0]), [(at + 1, 0)], {}
        while written and todo:
            i, waited = todo.pop()
            while i < len(code) and waited < need and seen.get(i, need) > waited:
                seen[i] = waited
                name, more = code[i]
                if more is not None:
                    if name.startswith("buffer_load") and more.endswith(" lds") and scalars(more) & written:
                        bad.append((f"{op} {args}", f"{name} {more}", waited))
                    if name == "s_endpgm":
                        break
                    waited += int(more) + 1 if name == "s_nop" else 1
                    if name == "s_branch":
                        i = label[more.strip()]
                        continue
                    if name.startswith("s_cbranch"):
                        todo.append((label[more.strip()], waited))
                i += 1
    return bad


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    b, folder = builder(), tmp_path_factory.mktemp("asm")
    if not os.path.exists(b.hipcc()):
        pytest.skip("hipcc not found")

    def build(source):
        out = str(folder / (source + ".s"))
        subprocess.run([b.hipcc(), *b.HIPCC_FLAGS, "--offload-device-only", "-S", os.path.join(b.CSRC, source), "-o", out],
                       check=True, capture_output=True)
        with open(out) as f:
            return kernels(f.read())

    with concurrent.futures.ThreadPoolExecutor() as pool:
        return dict(zip(("fwd", "bwd"), pool.map(build, ("dwattn_fwd.hip", "dwattn_bwd.hip"))))


def test_the_check_itself():
    ok = [(PRODUCT, "v[0:15], v[16:19], v[20:23], 0"), (PRODUCT, "v[0:15], v[16:19], v[20:23], v[0:15]"), ("s_nop", "11"),
          ("v_add_f32_e32", "v30, v3, v31"), ("s_endpgm", "")]
    assert too_early(ok) == []
    assert len(too_early(ok[:2] + [("s_nop", "10")] + ok[3:])) == 1
    assert len(too_early(ok[:1] + [(PRODUCT, "v[32:47], v[14:17], v[20:23], 0")] + ok[2:])) == 1
    # two ways to the read, the shorter one too short
    fork = ok[:2] + [("s_cbranch_scc1", ".LBB0_1"), ("s_nop", "9"), ("s_nop", "0"), (".LBB0_1", None), *ok[3:]]
    assert [w for _, _, w in too_early(fork)] == [1]


@pytest.mark.parametrize("which", ["fwd", "bwd"])
def test_results_are_read_after_their_wait(assembly, which):
    found = {name: too_early(code) for name, code in assembly[which].items()}
    assert sum(op == PRODUCT for code in assembly[which].values() for op, _ in code) > 1000
    assert not any(found.values()), {n: b[:2] for n, b in found.items() if b}


@pytest.mark.parametrize("which", ["fwd", "bwd"])
def test_m0_is_the_direct_loads_own(assembly, which):
    others = [(op, args) for code in assembly[which].values() for op, args in code
              if args and re.search(r"\bm0\b", args) and not (op == "s_mov_b32" and args.startswith("m0"))]
    assert not others, others[:3]


@pytest.mark.parametrize("which", ["fwd", "bwd"])
def test_direct_loads_keep_clear_of_their_scalars(assembly, which):
    early = [("v_readfirstlane_b32", "s4, v0"), ("s_mov_b32", "m0, s9"), ("s_nop", "0"),
             ("buffer_load_dwordx4", "v1, s[4:7], 0 offen lds")]
    assert len(loads_too_early(early)) == 1 and not loads_too_early(early[:1] + [("s_nop", "2")] + early[1:])
    loads = [args for code in assembly[which].values() for op, args in code if op.startswith("buffer_load") and args.endswith(" lds")]
    assert len(loads) > 100
    found = {name: loads_too_early(code) for name, code in assembly[which].items()}
    assert not any(found.values()), {n: b[:2] for n, b in found.items() if b}
