"""The example of README.md that attends over whole prompts and forks a session, run as written (seeded)."""
import math
import os
import re

import pytest
import torch

from paged_kv_decode_block_gb300 import pkv

pytestmark = pytest.mark.gpu


def test_readme_extend_example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.manual_seed(0)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "README.md")) as f:
        examples = re.findall(r"```python\n(.*?)```", f.read(), re.S)[:3]
    s = {}
    for example in examples:
        exec(example, s)
    torch.cuda.synchronize()
    assert s["plan"].status() == 0
    # the last tokens' attention is what the decode of the example before gave, each within its roundings
    last = s["attended"][s["cu"][1:].long() - 1].float()
    assert ((last - s["out"]).abs() <= 2.0 ** -7 * s["out"].abs() + 2.0 ** -9).all()
    # a token in the middle, in 64 bits from the cache
    t, b = 1017, 1                     # token 17 of the second row
    n = torch.arange(18, device="cuda")
    flat = s["table"][b].long()[n // 16] * 16 + n % 16
    k, v = (x.flatten(0, 1).view(torch.uint8)[flat].view(torch.float8_e4m3fn).double() * c.flatten(0, 1)[flat // 16][..., None].double()
            for x, c in ((s["k8"], s["ks"]), (s["v8"], s["vs"])))
    for h in range(32):
        w = torch.softmax(k[:, h // 4] @ s["q_new"][t, h].double() / math.sqrt(128), 0)
        ref, size = w @ v[:, h // 4], w @ v[:, h // 4].abs()
        assert ((s["attended"][t, h].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -10 * size).all()
    # the forks: what they hold is the prompt's
    for row, m in zip(s["two"], (1000, 500)):
        i = torch.arange(m, device="cuda")
        mine, his = (tab.long()[i // 16] * 16 + i % 16 for tab in (row, s["table"][0]))
        for x in ("k8", "v8"):
            pool = s[x].flatten(0, 1).view(torch.uint8)
            assert torch.equal(pool[mine], pool[his])
        for x in ("ks", "vs"):
            pool = s[x].flatten(0, 1)
            assert torch.equal(pool[mine // 16], pool[his // 16])
    assert s["copies"].tolist() == [[62, 66, 8], [31, 67, 4]] and s["pool"].free_count() == 60
