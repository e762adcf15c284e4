"""LDS reads that may still be on their way when a wave signals a barrier, from
the gfx950 assembly of a HIP source.

Waves that pass the barrier may overwrite what such a read has not fetched yet:
an s_barrier waits for nothing by itself.  LDS operations of a wave end in order,
so behind `s_waitcnt lgkmcnt(n)` at most the last n are under way.  Followed over
every path of a kernel: how many operations were issued since the oldest read or
write of LDS that no wait has covered (0: none)."""
from __future__ import annotations

import re

_LABEL = re.compile(r"^([.\w$]+):")
_WAIT = re.compile(r"lgkmcnt\((\d+)\)")
# Exchanges between lanes run through the LDS unit but touch no LDS.
_EXCHANGE = ("ds_bpermute", "ds_permute", "ds_swizzle")
_MOST = 16  # lgkmcnt counts to 15


def _kernels(asm: str):
    """(name, instructions and labels) of every kernel."""
    name, body = None, []
    kernels = set(re.findall(r"^\s*\.amdhsa_kernel\s+(\S+)", asm, re.M))
    for line in asm.splitlines():
        line = line.split(";")[0].strip()
        m = _LABEL.match(line)
        if m and m.group(1) in kernels:
            name, body = m.group(1), []
        elif name is None or not line:
            continue
        elif m:
            body.append(line)
            if m.group(1).startswith(".Lfunc_end"):
                yield name, body
                name = None
        elif not line.startswith("."):
            body.append(line)


def _after(line: str, n: int) -> int:
    op = line.split()[0]
    if op == "s_waitcnt":
        m = _WAIT.search(line)
        if m:
            return min(n, int(m.group(1)))
        return 0 if line.split()[1:] == ["0"] else n
    counts = op.startswith(("ds_", "s_load", "s_buffer_load"))
    begins = op.startswith("ds_") and not op.startswith(_EXCHANGE)
    return min(n + 1, _MOST) if begins or (counts and n) else n


def barriers(asm: str):
    """{kernel: [operations that may be under way at each s_barrier]}"""
    out = {}
    for name, body in _kernels(asm):
        at = {_LABEL.match(l).group(1): i for i, l in enumerate(body)
              if _LABEL.match(l)}
        state = [-1] * (len(body) + 1)
        todo = [(0, 0)]
        while todo:
            i, n = todo.pop()
            while i < len(body) and n > state[i]:
                state[i] = n
                line = body[i]
                if _LABEL.match(line):
                    i += 1
                    continue
                op = line.split()[0]
                if op == "s_endpgm":
                    break
                if op == "s_setpc_b64":
                    raise ValueError(f"{name}: {line}: a path that is not known")
                # A called function waits for everything before it begins.
                n = 0 if op == "s_swappc_b64" else _after(line, n)
                if op == "s_branch":
                    i = at[line.split()[1]]
                    continue
                if op.startswith("s_cbranch"):
                    todo.append((at[line.split()[1]], n))
                i += 1
        out[name] = [state[i] for i, l in enumerate(body)
                     if l.split()[0] == "s_barrier"]
    return out
