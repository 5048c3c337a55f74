"""What the compiler makes of the MXFP4 kernels: the device code is built to assembly and read."""
import os
import re
import subprocess

import pytest

from mask_only_logits_amd import build


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    try:
        hipcc = build.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not found")
    out = str(tmp_path_factory.mktemp("code") / "gemm_mxfp4.s")
    subprocess.run([hipcc, *build.HIPCC_FLAGS, "-I", str(build.ROOT / "include"), "-S", "--cuda-device-only",
                    str(build.CSRC / "gemm_mxfp4.hip"), "-o", out], check=True, stderr=subprocess.DEVNULL)
    with open(out) as f:
        text = f.read()
    os.remove(out)
    return text


def _arguments(text, kernel):
    """For each instance of a kernel: its arguments, as {offset: description} of the code object's metadata."""
    found = {}
    for block in re.split(r"^  - ", text[text.index("amdhsa.kernels:"):], flags=re.M)[1:]:
        name = re.search(r"\.symbol:\s+(\S+)\.kd", block)
        if name and kernel in name.group(1):
            args = re.split(r"^      - ", block[block.index(".args:"):], flags=re.M)[1:]
            at = [(re.search(r"\.offset:\s+(\d+)", a), a) for a in args]
            found[name.group(1)] = {int(o.group(1)): a for o, a in at if o}
    return found


def test_rows_may_be_quantized_in_place(assembly):
    # X (the first argument) and values (the last before the launch's own) may be one array: the compiler must not
    # take X for data that the kernel leaves alone, as it does of a pointer that nothing else may alias
    kernels = _arguments(assembly, "quantize_mxfp4_kernel")
    assert len(kernels) == 2
    for name, args in kernels.items():
        assert "global_buffer" in args[0] and "actual_access" not in args[0], name
        pointers = [o for o in sorted(args) if "global_buffer" in args[o]]
        assert len(pointers) == 5 and "actual_access" not in args[pointers[-1]], name


def _small_forms(text):
    """Template arguments (BM, BV, WGM, NSTAGE, STREAM, WORDS, OUT_BF16) of the small product kernels, and their names."""
    names = set(re.findall(r"^(_ZN\S*gemm_mxfp4_small_kernel\S*):", text, flags=re.M))
    return {tuple(int(x) for x in re.findall(r"L[ib](\d+)E", n)): n for n in names}


def test_no_form_is_built_that_no_call_takes(assembly):
    # five forms with scales by words or by bytes, and two that only scale rows of no whole words take, for either type
    forms = _small_forms(assembly)
    assert len(forms) == 2 * (5 * 2 + 2)
    for f in forms:
        assert f[:2] not in ((64, 128), (128, 128)) or f[5] == 0, f


def _requests(text, name):
    """What a kernel asks of memory, in the assembly's order: s a load of scales to a register, L a request to LDS, W n a
    wait for all but n of them, | a barrier, and a space where its blocks of instructions end."""
    body = text[text.index(f"\n{name}:"):]
    body = body[:body.index(".Lfunc_end")]
    found = []
    for line in body.splitlines():
        line = line.strip()
        wait = re.match(r"s_waitcnt\b.*vmcnt\((\d+)\)", line)
        if wait:
            found.append(f"W{wait.group(1)} ")
        elif line.startswith("s_barrier"):
            found.append("| ")
        elif line.startswith("global_load_lds"):
            found.append("L")
        elif re.match(r"(global|flat|buffer|scratch)_load", line):
            found.append("s")
        elif re.match(r"s_c?branch|\.LBB", line):
            found.append(" ")
    return re.sub(r" +", " ", "".join(found))


def test_counted_waits_of_the_small_tiles(assembly):
    """A step waits until all but the requests of the K tiles behind its own have come.  That counts each K tile's loads
    and requests, so the compiler must leave their number and order: NSTAGE - 1 K tiles before the first barrier, one
    after each, and nothing else."""
    forms = _small_forms(assembly)
    assert forms
    for (bm, bv, wgm, nstage, _, words, _), name in forms.items():
        tile = "s" * ((bv // (4 // wgm) // 16 + bm // wgm // 16) * (1 if words else 2)) + "L" * (bv // 32 + bm // 32)
        steps = _requests(assembly, name).split("|")
        assert len(steps) == nstage + 1, name
        first = [w for w in steps[0].split() if w != "W0"]
        assert first == [tile] * (nstage - 1) + [f"W{(nstage - 2) * len(tile)}"], name
        for k, step in enumerate(steps[1:]):
            want = [tile, f"W{(nstage - 2) * len(tile)}" if k < nstage - 1 else "W0"]
            assert step.split() == want, name


def test_counted_waits_of_the_large_tiles(assembly):
    """An output tile's first wait leaves its second K tile's codes under way: 12 requests (128 rows) or 16 a wave, which
    have to be the last of the prologue, behind all others."""
    names = sorted(set(re.findall(r"^(_ZN\S*gemm_mxfp4_kernel\S*):", assembly, flags=re.M)))
    assert len(names) == 2 * 2 * 3
    for name in names:
        bm, _, _, grouped = (int(x) for x in re.findall(r"L[ib](\d+)E", name))
        codes = 8 + bm // 32
        scales = 6 if grouped else 3 * (2 + bm // 128)
        seen = _requests(assembly, name)
        assert f" {'L' * (scales + codes)} {'L' * codes} W0 W{codes} | " in seen, name
        assert not re.search(rf"W{codes} (?!\|)", seen), name
