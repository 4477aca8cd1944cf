"""README.md's example of the 4-bit cache, run as it stands."""
import os
import re

import numpy as np
import pytest

from tests.gpu_common import ensure_built

pytestmark = pytest.mark.gpu


def test_example_of_the_4_bit_cache():
    # operands cut from one projection, and heads-major ones (transposed
    # views): the same outputs; a sequence without a new token keeps its own
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()
    import certified_sparse_attention_gb300 as csa
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    made, = [b for b in blocks if "csa.QKNormRope(" in b]
    used, = [b for b in blocks if "csa.KV4Cache(" in b]
    dev = "cuda"
    rng = np.random.default_rng(3)

    def bf16(*size):
        return torch.from_numpy(rng.normal(size=size).astype(np.float32)).to(dev).bfloat16()
    B, T, Hq, Hkv, d, n_max = 2, 1, 8, 2, 128, 256
    qkv = bf16(B, T, Hq + 2 * Hkv, d)
    side = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    major = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in side]
    # two tokens, heads-major: their rows' strides are not those of [B][T][Hkv][d]
    two = [x.repeat(1, 2, 1, 1).transpose(1, 2).contiguous().transpose(1, 2) for x in side]
    w = bf16(d)
    out = []
    for (q, k, v), new in ((side, [1, 0]), (major, [1, 0]), (two, [2, 1])):
        T = q.shape[1]
        ns = dict(torch=torch, csa=csa, wq=w, wk=w, inv_freq=10000.0 ** (-np.arange(64) / 64),
                  shape=csa.make_shape(B, Hq, Hkv, d, n_max, "bf16"), q=q, k=k, v=v,
                  lens_dev=torch.tensor([2, 1], dtype=torch.int64, device=dev),
                  n_new=torch.tensor(new, dtype=torch.int64, device=dev),
                  first=torch.zeros(B, dtype=torch.int64, device=dev))
        ns["K"], ns["V"], ns["K16"], ns["V16"] = [
            torch.zeros(B, Hkv, n_max, d, dtype=torch.bfloat16, device=dev) for _ in range(4)]
        exec(made, ns)
        exec(used.replace("T=1)", f"T={T})"), ns)
        assert csa.csa_check(ns["attend"].ws) == 0 and csa.csa_check(ns["cache"].refused) == 0
        o = ns["o"]
        for b in range(B):
            assert bool((o[b, new[b]:] == 0).all()) and bool((o[b, :new[b]] != 0).all())
        out.append(o.clone())
    assert torch.equal(out[0], out[1])
