"""README.md's example of the 8-bit cache, run as it stands."""
import os
import re

import numpy as np
import pytest

from tests.gpu_common import ensure_built

pytestmark = pytest.mark.gpu


def test_example_of_the_8_bit_cache():
    # Operands cut from one projection, and heads-major ones (transposed views): the
    # same outputs.  A sequence's rows past its new tokens keep their zeros.  With 8
    # blocks at most, everything is chosen.
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()
    import certified_sparse_attention_gb300 as csa
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    used, = [b for b in blocks if "csa.KV8Cache(" in b]
    rng = np.random.default_rng(4)
    B, T, Hq, Hkv, d, n_max = 2, 300, 8, 2, 128, 512
    # (16 new tokens at most attend at once: the prompt goes in first)
    qkv = torch.from_numpy(rng.normal(size=(B, T, Hq + 2 * Hkv, d)).astype(np.float32)).cuda().bfloat16()
    new = 3
    out = []
    for major in (False, True):
        parts = [qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]]
        if major:
            parts = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in parts]
        shape = csa.make_shape(B, Hq, Hkv, d, n_max, "bf16")
        prompt = csa.KV8Cache(shape, "cuda")
        n0 = torch.tensor([T - new, 70], dtype=torch.int64, device="cuda")
        prompt.append(parts[1][:, :T - new], parts[2][:, :T - new], n0, n0)
        held = [getattr(prompt, name) for name, _, _ in prompt._layout(B, Hkv, n_max // 64, d)]
        # the example's cache is the prompt's, one token more of it in sequence 1
        code = used.replace('csa.KV8Cache(shape, "cuda")', 'csa.KV8Cache(shape, "cuda", held)')
        assert code != used
        q, k, v = [x[:, T - new:] for x in parts]
        n_new = torch.tensor([new, 1], dtype=torch.int64, device="cuda")
        ns = dict(torch=torch, csa=csa, shape=shape, T=new, q=q, k=k, v=v, lens_dev=n0 + n_new, n_new=n_new, held=held)
        exec(code, ns)
        for x in (ns["dense"].ws, ns["sparse"].ws, ns["sparse"].status):
            assert csa.csa_check(x) == 0
        o = ns["o"]
        assert bool((o[1, 1:] == 0).all()) and bool((o[0] != 0).all()) and bool((o[1, :1] != 0).all())
        # everything chosen, the blocks up to each token's own
        assert ns["count"][0, :, 0].tolist() == [5, 5, 5] and ns["count"][1, 0].tolist() == [2, 2]
        # Both sum the same terms, grouped otherwise.  A score's terms are below 32 in all
        # (in magnitude, base 2), of which 2^-22 is lost and float32's roundings: each weight
        # is within 1e-5 of itself, and the outputs, weighted means of |values| < 6, within
        # 2 * 1e-5 * 6 of each other.
        for other in (ns["o_sparse"], ns["o_lists"]):
            assert float((o - other).abs().max()) < 1.2e-4
        assert torch.equal(ns["o_sparse"], ns["o_lists"])
        out.append(o.clone())
    assert torch.equal(out[0], out[1])
