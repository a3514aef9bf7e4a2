"""The 8-bit cache example of README.md, run as written (seeded), against the fp64 oracle: the decode
over the cache as the device holds it, and the cache against the definitions (a code is off by at
most half an e4m3 step of its value or of the subnormal range)."""
import os
import re

import numpy as np
import pytest
import torch

from oracle import cache8
from paged_kv_decode_block_gb300 import pkv

pytestmark = pytest.mark.gpu


def test_readme_cache8_example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.manual_seed(0)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "README.md")) as f:
        first, second = re.findall(r"```python\n(.*?)```", f.read(), re.S)[:2]
    space = {}
    exec(first, space)
    exec(second.replace("qkv = torch.randn", "qkv = QKV = torch.randn").replace("pkv.append_q8", "QKV = QKV.clone(); pkv.append_q8"),
         space)
    torch.cuda.synchronize()
    s = space
    assert s["plan"].status() == 0 and s["after"].tolist() == s["lens_h"]
    codes = [s[x].view(torch.uint8).cpu().numpy() for x in ("k8", "v8")]
    scales = [s[x].cpu().numpy() for x in ("ks", "vs")]
    table = s["table_h"].numpy()
    to64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    out, lse = cache8.decode_q8(to64(s["q_last"]), *codes, *scales, table, s["lens_h"])
    # 1000 tokens: 2e-3 on out and 1e-4 on lse, the decode's tolerances
    assert np.max(np.abs(s["out"].cpu().numpy() - out)) <= 2e-3
    assert np.max(np.abs(s["lse"].cpu().numpy() - lse)) <= 1e-4
    before = to64(s["QKV"])   # the projection before the queries turned in place
    freq = 10000.0 ** (-np.arange(0, 128, 2) / 128)
    t = 0
    for b, n in enumerate(s["lens_h"]):
        rows = cache8.places(table, b, 0, n, 16)
        for x, c, sc in ((cache8.rotate(before[t:t + n, 32:40], np.arange(n), freq), codes[0], scales[0]),
                         (before[t:t + n, 40:], codes[1], scales[1])):
            size = sc.reshape(-1, 8)[rows // 16].astype(np.float64)[..., None]
            got = cache8.E4M3[c.reshape(-1, 8, 128)[rows]] * size
            assert np.all(np.abs(got - x) <= 2.0 ** -4 * np.abs(x) + size * 2.0 ** -10 + 2.0 ** -20 * 2 * np.abs(x).max())
        t += n
