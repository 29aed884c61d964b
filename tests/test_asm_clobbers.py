"""CPU check of the inline assembly in the sources: a fixed register that a statement writes is
named among its clobbers, so that the compiler keeps nothing of its own there."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = sorted(glob.glob(os.path.join(ROOT, "allreduce_reduction_nranks_amd", "csrc", "*")))


def statements(text):
    """Bodies of the asm statements, parentheses balanced outside of strings."""
    for m in re.finditer(r"\basm\s+(?:volatile\s*)?\(", text):
        depth, at, quoted = 1, m.end(), False
        while depth:
            c = text[at]
            if c == '"' and text[at - 1] != "\\":
                quoted = not quoted
            elif not quoted:
                depth += (c == "(") - (c == ")")
            at += 1
        yield text[m.end():at - 1]


def parts(body):
    """(template, clobbers) of a statement."""
    fields, at, quoted = [""], 0, False
    for k, c in enumerate(body):
        if c == '"' and body[k - 1] != "\\":
            quoted = not quoted
        if c == ":" and not quoted:
            fields.append("")
        else:
            fields[-1] += c
    template = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', fields[0])).replace("\\n", "\n").replace("\\t", " ")
    return template, re.findall(r'"([^"]*)"', fields[3]) if len(fields) > 3 else []


def test_written_registers_are_clobbered():
    seen = 0
    for path in SOURCES:
        for body in statements(open(path).read()):
            template, clobbers = parts(body)
            seen += 1
            for line in re.split(r"[\n;]", template):
                words = line.split(None, 1)
                if len(words) < 2 or words[0].startswith(("s_waitcnt", "s_cmp", "s_barrier")):
                    continue
                to = words[1].split(",")[0].strip()
                if to in ("m0", "vcc", "exec", "scc") or re.fullmatch(r"[sv](\d+|\[\d+:\d+\])", to):
                    assert to in clobbers, "%s: %r writes %s" % (os.path.basename(path), line.strip(), to)
    assert seen >= 4
