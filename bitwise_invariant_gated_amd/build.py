"""Build libgdn_cpr.so in-tree for gfx950 with hipcc.

    python -m bitwise_invariant_gated_amd.build

Flags that fix the numerics: -ffp-contract=off (every FMA in the library is
written explicitly), no fast-math, and packed-fp32 instructions disabled for
the device code.
"""

from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRCS = [os.path.join(HERE, "csrc", n) for n in ("gdn_cpr.hip", "gdn_attn.hip")]
OUT = os.path.join(HERE, "libgdn_cpr.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    "-ffp-contract=off",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


def check_dpp_hazards(asm_text: str) -> list:
    """Every v_fmac_f32_dpp must not read, as its DPP source, a VGPR that a
    VALU instruction wrote within the two preceding wait states (the gfx9
    VALU-write -> DPP-read hazard; s_nop N provides N + 1 wait states).
    Returns a list of violations (function, line number, text)."""
    import re
    bad = []
    func = "?"
    recent = []  # (wait states it provides, set of VGPRs it wrote)
    vreg = re.compile(r"^v(\d+)$|^v\[(\d+):(\d+)\]$")

    def regs(tok):
        m = vreg.match(tok.strip())
        if not m:
            return set()
        if m.group(1) is not None:
            return {int(m.group(1))}
        return set(range(int(m.group(2)), int(m.group(3)) + 1))

    for no, line in enumerate(asm_text.splitlines(), 1):
        t = line.strip()
        if not t or t.startswith(";") or t.startswith("."):
            continue
        if t.endswith(":"):
            if not t.startswith(".L"):
                func = t[:-1]
                recent = []
            continue
        parts = t.split(None, 1)
        op = parts[0]
        args = [a.strip() for a in parts[1].split(",")] if len(parts) > 1 else []
        if "_dpp" in op and len(args) >= 2:  # the DPP source is src0
            src = regs(args[1].split()[0])
            waits = 0
            for ws, wrote in reversed(recent):
                if waits >= 2:
                    break
                if wrote & src:
                    bad.append((func, no, t))
                    break
                waits += ws
        if op == "s_nop":
            ws = int(args[0], 0) + 1 if args else 1
            recent.append((ws, set()))
        elif op.startswith("v_") and args:
            first = args[0].split()[0]
            recent.append((1, regs(first) if not first.startswith("s") else set()))
        else:
            recent.append((1, set()))
        recent = recent[-4:]
    return bad


# kernels on the bf16 hot paths (prefill, decode, continuation, fwd_bwd, and the
# attention layer), by mangled-name fragment; register spills there cost a
# scratch set-up per launch and memory traffic per spill, so the build rejects them
HOT_KERNELS = ("k_scanIN3cpr4Bf16", "k_chain_scan_bf16", "k_decodeIN3cpr4Bf16", "k_resync_bf16",
               "k_cont_headIN3cpr4Bf16", "k_chunk_local_prefill_bf16", "k_chain_prefill_bf16", "k_bwd_local_bf16",
               "k_bwd_chain_bf16", "k_bwd_state_grads_bf16", "k_plan", "k_attn_")

# three of them fill the registers, and spill: up to this many.  k_attn_prefill
# reloads one value beside the score MFMAs of a tile, and its fold at the end of a partition
# stores and reloads 14 (d = 128) or one (256); k_attn_rows of two row tiles at d = 128
# reloads one or two in each part of its loop
MAY_SPILL = {"k_attn_prefillILi128E": 76, "k_attn_prefillILi256E": 21, "k_attn_rowsILi128ELi2E": 14}


def check_spills(asm_text: str, hot=HOT_KERNELS, may=MAY_SPILL) -> list:
    """(kernel, spilled VGPRs) for every hot kernel whose metadata records
    more VGPR spills than it may have."""
    import re
    bad = []
    for m in re.finditer(r"\.name:\s+(\S+)\n(.*?)\.wavefront_size", asm_text, re.S):
        name, body = m.group(1), m.group(2)
        sp = re.search(r"\.vgpr_spill_count:\s+(\d+)", body)
        most = next((n for frag, n in may.items() if frag in name), 0)
        if sp and int(sp.group(1)) > most and any(h in name for h in hot):
            bad.append((name, int(sp.group(1))))
    return bad


def check_isa(texts: list, verbose: bool = True) -> None:
    """Check the sources' device assembly: the DPP hazard rule, and that no
    hot kernel spills (or more than it may)."""
    n_dpp = sum(t.count("v_fmac_f32_dpp") for t in texts)
    bad = [v for t in texts for v in check_dpp_hazards(t)]
    if bad:
        raise RuntimeError(f"DPP hazard in generated code ({len(bad)}): " + "; ".join(
            f"{fn} line {no}: {t}" for fn, no, t in bad[:5]))
    spills = [v for t in texts for v in check_spills(t)]
    if spills:
        raise RuntimeError("register spills in hot kernels: " + "; ".join(f"{n} ({k})" for n, k in spills))
    if verbose:
        print(f"ISA check: {n_dpp} v_fmac_f32_dpp instructions, no VALU-write -> DPP-read hazard, "
              "no spills in the hot kernels beyond those listed")


def _run(cmds: list) -> str:
    """Run the compiler commands side by side; their messages."""
    procs = [subprocess.Popen(c, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True) for c in cmds]
    outs = [p.communicate()[0] for p in procs]
    # the host pass does not know the packed-fp32 target feature; that warning is expected
    lines = [ln for o in outs for ln in o.splitlines() if "packed-fp32-ops" not in ln
             and ln.strip() and not ln.startswith("1 warning")]
    bad = [p.returncode for p in procs if p.returncode != 0]
    if bad:
        sys.stderr.write("\n".join(lines) + "\n")
        raise RuntimeError(f"hipcc failed with status {bad[0]}")
    return "\n".join(lines)


def build(verbose: bool = True) -> str:
    """Objects and device assembly of every source, side by side, then the link."""
    import tempfile
    tmp = OUT + ".tmp"
    with tempfile.TemporaryDirectory() as d:
        stem = [os.path.join(d, os.path.basename(s)) for s in SRCS]
        base = [f for f in FLAGS if f != "-shared"]
        cmds = [[HIPCC, *base, "-c", "-o", o + ".o", s] for s, o in zip(SRCS, stem)]
        cmds += [[HIPCC, *[f for f in base if f != "-fPIC"], "--cuda-device-only", "-S", "-o", o + ".s", s]
                 for s, o in zip(SRCS, stem)]
        if verbose:
            print("\n".join(" ".join(c) for c in cmds[:len(SRCS)]), flush=True)
        said = _run(cmds)
        if verbose and said:
            print(said)
        _run([[HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *[o + ".o" for o in stem]]])
        texts = []
        for o in stem:
            with open(o + ".s") as f:
                texts.append(f.read())
    check_isa(texts, verbose)
    os.replace(tmp, OUT)
    return OUT


if __name__ == "__main__":
    build()
