"""The waits of kernels that stand in headers: one answer for all lanes of a warp."""
import glob
import os
import re

from test_warp_waits import CSRC


def text(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def kernels():
    """(file, text) of every kernel of a header in which a lane elected of a whole warp issues."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cuh"))):
        name = os.path.basename(path)
        for part in re.split(r"^__global__", text(name), flags=re.M)[1:]:
            body = part.split("\n}\n")[0]
            if "elect_one()" in body:
                yield name, body


def test_warp_wide_loops_wait_with_one_answer():
    """elect.sync needs every lane at the same place: waits and looks at barriers are voted on, drains are one lane's."""
    found = list(kernels())
    assert {f for f, _ in found} == {"w4_tc.cuh"}
    for name, body in found:
        code = [line.split("//")[0] for line in body.splitlines()]
        assert sum("wait_warp(" in line for line in code) >= 8  # every role
        for line in code:
            assert not re.search(r"\b(mbar_wait|mbar_try_wait)\(", line), (name, line)
        # looks without a wait: `seen` alone, whose answer is voted on before it counts
        looks = [line for line in code if "mbar_test(" in line]
        assert len(looks) == 1 and "auto seen" in looks[0]
        assert [line.strip() for line in code if "seen(" in line] == ["const bool look = seen(after);"]
        assert [line.strip() for line in code if re.search(r"\blook\b", line)][1:] == ["ready = __all_sync(0xffffffffu, look);"]
        # the issuer's wait for operands is made of voted ones
        waits = "".join(code).split("auto wait_for =")[1].split("};")[0]
        assert waits.count("wait_warp(") == 2
    for line in text("w4_tc.cuh").splitlines():
        if "mbar_drain(" in line:
            assert "lane == 0" in line or "mbar_drain(&sh.cfull" in line or "mbar_drain(&sh.xfull" in line, line


def test_the_poll_is_voted_on():
    body = text("w4_tc.cuh").split("bool wait_warp(")[1].split("\n}\n")[0]
    assert "__all_sync(0xffffffffu, mbar_try_wait(bar, parity))" in body and "return mbar_wait_warp(" in body
    assert body.count("mbar_try_wait(") == 1
