"""Values read from tensor memory are there only after the wait (host: held in the source, since a compiler that moved a
use above the wait would show on a GPU as now and then a wrong result). The wait names no register: a load's results are
bound to it by standing in the same statement, or by a statement behind it that takes and gives back every register."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fully_sharded_gb300", "csrc")
LOAD, WAIT = "tcgen05.ld.", "tcgen05.wait::ld"


def statements(source):
    """(start, text) of each asm statement."""
    for m in re.finditer(r"\basm\b(?: volatile)?\(", source):
        depth, end, quoted = 1, m.end(), False
        while depth:
            c = source[end]
            if c == '"' and source[end - 1] != "\\":
                quoted = not quoted
            elif not quoted:
                depth += {"(": 1, ")": -1}.get(c, 0)
            end += 1
        yield m.start(), source[m.start():end]


def unbound(source):
    """The loads whose results nothing binds to the wait."""
    found = list(statements(source))
    bad = []
    for k, (at, load) in enumerate(found):
        if LOAD not in load or load.find(WAIT) > load.find(LOAD):
            continue
        function = source.index("\n}", at)  # the end of the function
        behind = [s for a, s in found[k + 1:] if a < function]
        waits = [i for i, s in enumerate(behind) if WAIT in s]
        taken = [m for s in behind[waits[0] + 1:] for m in re.findall(r'"\+r"\((\w+)\[', s)] if waits else []
        bad += [w for w in re.findall(r'"=r"\((\w+)\[', load) if w not in taken][:1]
    return bad


def test_every_load_is_bound_to_its_wait():
    loads = 0
    for name in sorted(os.listdir(CSRC)):
        source = open(os.path.join(CSRC, name)).read()
        assert unbound(source) == [], name
        loads += source.count(LOAD)
    assert loads >= 2


def test_a_loose_load_is_seen():
    loose = """void f() {
  asm volatile("tcgen05.ld.sync {%0}, [%1];" : "=r"(r[0]) : "r"(a));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  use(r[0]);
}
"""
    assert unbound(loose) == ["r"]
    assert unbound(loose.replace("  use", '  asm volatile("" : "+r"(r[0]));\n  use')) == []
    assert unbound(loose.replace(";\" : \"=r\"", ";\\n tcgen05.wait::ld.sync.aligned;\" : \"=r\"")) == []
