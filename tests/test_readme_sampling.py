"""The README's steps draw noise of their own for every token: run over batches and trees that change from step to step, its
sampling lines use no row of the noise (row + offset of one seed) twice."""
import os
import re

import pytest

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def sampling_lines():
    """Of each Python block that samples: the lines that do, and what they need of the block's own count of rows."""
    with open(README) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    for block in blocks:
        lines = [line for line in block.splitlines() if not line.startswith("#")]
        count = [line for line in lines if re.match(r"drawn\b", line)]
        for line in lines:
            if "pkv.pkv_sample" in line:
                yield line, count


CASES = list(sampling_lines())


class Recorder:
    def __init__(self):
        self.rows = []

    def pkv_sample(self, logits, *rest, seed, offset):
        self.rows += [(seed, offset + i) for i in range(len(logits))]
        return list(range(len(logits)))

    pkv_sample_filtered = pkv_sample


def test_the_lines_are_found():
    assert {re.search(r"pkv_sample\w*\((\w+)", line).group(1) for line, _ in CASES} == {"logits", "logits_t"}


@pytest.mark.parametrize("line,count", CASES, ids=[str(i) for i in range(len(CASES))])
def test_no_noise_twice(line, count):
    pkv = Recorder()
    names = {"pkv": pkv, "drawn": 0, **dict.fromkeys(("temperatures", "temperatures_t", "top_k", "top_p", "min_p"))}
    start = [x for x in count if re.match(r"drawn\s*=", x)]
    for x in start:
        exec(x, names)
    for step, rows in enumerate((20, 30, 1, 25, 20, 3)):
        names.update(step=step, batch=rows, nodes=rows, logits=[0.0] * rows, logits_t=[0.0] * rows)
        exec(line, names)
        for x in count:
            if x not in start:
                exec(x, names)
    assert len(set(pkv.rows)) == len(pkv.rows)
